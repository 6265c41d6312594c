"""CPU checks of the block-scaled cache's entry points: arguments that are
refused before anything is launched, the frequency tables, and the binding's
own checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

from fp8_paged_kv_attn_gb300 import kvq

INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 4


def block_cache(**kw):
    c = kvq.CBlockCache(16, 16, 16, 8, 16, 2, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rope_desc(**kw):
    r = kvq.CRope(16, 128, 0, 1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


ARGS = {
    "append": dict(k=16, ks=256, v=16, vs=256, ts=16, n=4, lens=16, bt=16, B=2, MP=4),
    "rope_append": dict(q=16, qs=512, qo=16, qos=512, Hq=4, k=16, ks=256, v=16, vs=256, ts=16, n=4,
                        lens=16, bt=16, B=2, MP=4),
    "read": dict(ts=16, n=4, first=16, bt=16, B=2, MP=4, k=16, ks=256, v=16, vs=256),
    "attn": dict(q=16, qs=512, Hq=4, ts=16, n=4, max_q=2, lens=16, bt=16, B=2, MP=4, mask=None,
                 sm=0.1, out=16, ws=256, wsb=1 << 40),
    "rope": dict(pos=16, n=4, D=128, q=16, qs=512, qo=16, qos=512, Hq=4, k=16, ks=256, ko=16,
                 kos=256, Hk=2),
}


def call(op, cache=None, rope=None, **kw):
    L = kvq.load()
    a = {**ARGS[op], **kw}
    assert set(a) == set(ARGS[op])
    c = ctypes.byref(cache if cache is not None else block_cache())
    r = ctypes.byref(rope if rope is not None else rope_desc())
    if op == "append":
        return L.kvq_block_append(c, *a.values(), None, None)
    if op == "rope_append":
        return L.kvq_rope_block_append(c, r, *a.values(), None, None)
    if op == "read":
        return L.kvq_block_read(c, *a.values(), None, None)
    if op == "attn":
        return L.kvq_block_attn(c, *a.values(), None, None)
    return L.kvq_rope(r, *a.values(), None)


@pytest.mark.parametrize("op", ["append", "rope_append", "read", "attn"])
@pytest.mark.parametrize("kw,want", [
    ({"k_pool": None}, INVALID), ({"v_pool": None}, INVALID), ({"scales": None}, INVALID),
    ({"k_pool": 8}, INVALID), ({"scales": 4}, INVALID), ({"num_pages": 0}, INVALID),
    ({"num_kv_heads": 0}, INVALID), ({"page_size": 8}, UNSUPPORTED),
    ({"page_size": 128}, UNSUPPORTED), ({"head_dim": 96}, UNSUPPORTED)])
def test_bad_cache(op, kw, want):
    assert call(op, cache=block_cache(**kw)) == want


BAD = [("append", k, v) for k, v in [("k", None), ("v", None), ("k", 8), ("v", 24), ("ks", 248),
                                     ("vs", 260), ("ks", 0), ("n", -1), ("B", -1), ("MP", 0),
                                     ("lens", None), ("bt", None), ("MP", 1 << 28)]]
BAD += [("rope_append", k, v) for k, v in [("q", None), ("qo", 8), ("qs", 504), ("qos", 516),
                                           ("Hq", -1), ("k", None), ("lens", None)]]
BAD += [("read", k, v) for k, v in [("k", None), ("v", 8), ("ks", 255), ("bt", None), ("n", -3)]]
BAD += [("attn", k, v) for k, v in [("q", None), ("q", 8), ("qs", 504), ("Hq", 3), ("Hq", 0),
                                    ("max_q", 0), ("max_q", 1 << 30), ("lens", None), ("bt", None),
                                    ("out", None), ("out", 8), ("ws", None),
                                    ("sm", math.inf), ("sm", math.nan), ("MP", 1 << 28)]]
BAD += [("rope", k, v) for k, v in [("pos", None), ("n", -1), ("q", None), ("qo", None), ("qs", 500),
                                    ("Hq", 0), ("Hk", -1), ("k", None), ("ko", 4), ("kos", 0)]]


@pytest.mark.parametrize("op,name,value", BAD)
def test_bad_arguments(op, name, value):
    assert call(op, **{name: value}) == INVALID


@pytest.mark.parametrize("op", ["rope_append", "rope"])
@pytest.mark.parametrize("kw", [{"inv_freq": None}, {"inv_freq": 4}, {"rotary_dim": 0},
                                {"rotary_dim": 24}, {"rotary_dim": 144}, {"layout": 2},
                                {"mscale": math.nan}])
def test_bad_rope(op, kw):
    assert call(op, rope=rope_desc(**kw)) == INVALID


def test_no_starts_means_one_row_a_request():
    for op in ("append", "read", "attn"):
        assert call(op, ts=None, n=3) == INVALID  # two requests
    assert call("rope", D=96) == UNSUPPORTED


def test_nothing_to_do_is_fine():
    for op in ("append", "rope_append", "read", "attn"):
        assert call(op, n=0) == 0
        assert call(op, B=0) == 0
    assert call("rope", n=0) == 0


def test_workspace_size_of_bad_shapes_is_zero():
    f = kvq.load().kvq_block_attn_workspace_size
    for a in ((-1, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 1, 7, 2, 128), (1, 1, 8, 0, 128),
              (1, 1, 8, 2, 96), (1, 1 << 30, 8, 2, 128)):
        assert f(*a) == 0


def test_inv_freq_plain_linear_and_base():
    f, m = kvq.kvq_rope_inv_freq(64)
    want = 10000.0 ** (-np.arange(32) / 32)
    assert m == 1.0 and np.allclose(f.numpy(), want, rtol=1e-14)
    g, _ = kvq.kvq_rope_inv_freq(64, scaling=kvq.ROPE_LINEAR, factor=8.0)
    assert np.allclose(g.numpy(), want / 8, rtol=1e-14)
    h, _ = kvq.kvq_rope_inv_freq(64, scaling=kvq.ROPE_BASE, factor=8.0)
    assert h[0] == 1.0 and math.isclose(h[-1], want[-1] / 8, rel_tol=1e-12)


@pytest.mark.parametrize("scaling", [kvq.ROPE_RAMP, kvq.ROPE_BANDS])
def test_inv_freq_mixed(scaling):
    rd, s, n, lo, hi = 128, 4.0, 8192.0, 1.0, 32.0
    f, m = kvq.kvq_rope_inv_freq(rd, 500000.0, scaling, s, n, lo, hi)
    f = f.numpy()
    plain = 500000.0 ** (-2.0 * np.arange(64) / rd)
    turns = n * plain / (2 * np.pi)
    # at the ends: kept above `high` turns, divided below `low`; monotone between
    margin = 500000.0 ** (2.0 / rd)  # one pair, for the ramp's rounded ends
    assert np.allclose(f[turns > hi * margin], plain[turns > hi * margin], rtol=1e-14)
    assert np.allclose(f[turns < lo / margin], plain[turns < lo / margin] / s, rtol=1e-14)
    assert (np.diff(f) < 0).all() and (f <= plain * (1 + 1e-14)).all() and (f >= plain / s * (1 - 1e-14)).all()
    assert math.isclose(m, 0.1 * math.log(s) + 1 if scaling == kvq.ROPE_RAMP else 1.0, rel_tol=1e-6)
    if scaling == kvq.ROPE_BANDS:
        keep = np.clip((turns - lo) / (hi - lo), 0, 1)
        assert np.allclose(f, plain / s * (1 - keep) + plain * keep, rtol=1e-12)


@pytest.mark.parametrize("args", [
    (0,), (24,), (64, 1.0), (64, math.inf), (64, 10000.0, 9), (64, 10000.0, 1, 0.5),
    (64, 10000.0, 3, 4.0, 0.0), (64, 10000.0, 4, 4.0, 4096.0, 0.0, 4.0),
    (64, 10000.0, 4, 4.0, 4096.0, 4.0, 4.0)])
def test_inv_freq_refusals(args):
    with pytest.raises(kvq.KvqError):
        kvq.kvq_rope_inv_freq(*args)


def test_binding_refuses_host_and_misshapen_tensors():
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        kvq.BlockKVCache(pool, pool, torch.ones(4, 2, 2))  # host memory
    with pytest.raises(ValueError):
        kvq.BlockKVCache(pool, pool[:2], torch.ones(4, 2, 2))
    with pytest.raises(ValueError):
        kvq.Rope(torch.zeros(8, dtype=torch.float64))
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for bad in (x, x.float(), x[:, :1], x.transpose(0, 1)):
        with pytest.raises(ValueError):
            kvq._rows(bad, "q", 3, 2, 64, 0)
    for bad in (torch.zeros(3, dtype=torch.int32), torch.zeros(3), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            kvq._arr(bad, "pos", (torch.int32,), (3,), 0)
