"""CPU checks of kvq_block_prefix_attn: arguments that are refused before anything is launched,
and the binding's checks."""
import ctypes
import math

import pytest
import torch

from fp8_paged_kv_attn_gb300 import kvq

INVALID, UNSUPPORTED = 1, 4
ARGS = dict(q=16, qs=512, Hq=4, ts=16, n=4, max_q=2, lens=16, bt=16, B=2, MP=4, gs=16, pp=16, groups=1, mask=None,
            sm=0.1, out=16, ws=256, wsb=1 << 40)


def call(cache=None, **kw):
    c = kvq.CBlockCache(16, 16, 16, 8, 16, 2, 128)
    for k, v in (cache or {}).items():
        setattr(c, k, v)
    a = {**ARGS, **kw}
    assert set(a) == set(ARGS)
    return kvq.load().kvq_block_prefix_attn(ctypes.byref(c), *a.values(), None, None)


@pytest.mark.parametrize("kw,want", [
    ({"k_pool": None}, INVALID), ({"v_pool": None}, INVALID), ({"scales": None}, INVALID), ({"v_pool": 8}, INVALID),
    ({"scales": 4}, INVALID), ({"num_pages": 0}, INVALID), ({"num_kv_heads": 0}, INVALID), ({"page_size": 8}, UNSUPPORTED),
    ({"page_size": 128}, UNSUPPORTED), ({"head_dim": 96}, UNSUPPORTED)])
def test_bad_cache(kw, want):
    assert call(cache=kw) == want


@pytest.mark.parametrize("name,value", [
    ("q", None), ("q", 8), ("qs", 504), ("qs", 516), ("Hq", 3), ("Hq", 0), ("Hq", -4), ("n", -1), ("max_q", 0),
    ("max_q", -1), ("lens", None), ("bt", None), ("B", -1), ("MP", 0), ("MP", 1 << 28), ("MP", (1 << 27) - 1),
    ("gs", None), ("pp", None), ("groups", -1), ("sm", math.inf), ("sm", math.nan), ("out", None), ("out", 8),
    ("ws", None)])
def test_bad_arguments(name, value):
    assert call(**{name: value}) == INVALID


def test_sizes_at_their_limits():
    assert call(ts=None, n=3) == INVALID  # two requests
    assert call(n=1 << 30, Hq=4) == INVALID  # rows times heads a kv head
    f = kvq.kvq_block_prefix_attn_workspace_size
    for a in ((-1, 8, 2, 128), (1, 7, 2, 128), (1, 0, 2, 128), (1, 8, 0, 128), (1, 8, 2, 96)):
        assert f(*a) == 0
    with pytest.raises(ValueError):
        kvq.block_prefix_workspace(4, 7, 2, 128, device="cpu")


def test_nothing_to_do_is_fine():
    none = dict(q=None, lens=None, out=None, ws=None, wsb=0, gs=None, pp=None)
    assert call(n=0, **none) == 0
    assert call(B=0, **none) == 0


def test_binding_wants_cuda_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pool = torch.zeros(8, 2, 16, 64, dtype=torch.uint8)
        cache = kvq.BlockKVCache(pool, pool, torch.ones(8, 2, 2))
        kvq.kvq_block_prefix_attn(cache, q, z[:3], z[:2], z.view(2, 2), z[:2], z[:1], torch.zeros_like(q), z)
