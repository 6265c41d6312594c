"""CPU checks of the calls for pages that several requests hold, and of page copies:
arguments that are refused before anything is launched, and the binding's checks."""
import ctypes

import pytest
import torch

from fp8_paged_kv_attn_gb300 import kvq

INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 4
BIG = 1 << 40

ARGS = {
    "fork": dict(stack=16, count=16, tags=16, shares=16, pages=8, table=16, expected=16, B=4, MP=4, P=16,
                 src=16, dst=16, tok=16, n=2, cs=16, cd=16, ok=16, ws=256, wsb=BIG),
    "release": dict(stack=16, count=16, shares=16, pages=8, table=16, B=4, MP=4, req=16, first=None, num=16,
                    n=2, ws=256, wsb=BIG),
    "compact": dict(stack=16, count=16, tags=16, shares=16, pages=9, table=16, expected=16, B=4, MP=4,
                    held=16, cs=16, cd=16, cap=4, moves=16, ws=256, wsb=BIG),
}


def call(op, **kw):
    a = {**ARGS[op], **kw}
    assert set(a) == set(ARGS[op])
    return getattr(kvq.load(), "kvq_pages_" + op)(*a.values(), None, None)


@pytest.mark.parametrize("op", ["fork", "release", "compact"])
def test_sizes_and_pointers(op):
    for name in ("pages", "B", "MP"):
        assert call(op, **{name: 0}) == INVALID
        assert call(op, **{name: -3}) == INVALID
    for name in ARGS[op]:
        if name in ("first", "ws") or not isinstance(ARGS[op][name], int) or ARGS[op][name] != 16:
            continue
        if name in ("P",):
            continue
        assert call(op, **{name: None}) == INVALID, name
    assert call(op, ws=None) == INVALID
    assert call(op, ws=272) == WORKSPACE
    need = kvq.kvq_pages_workspace_size(ARGS[op]["pages"], 4)
    assert need % 256 == 0 and need >= 4 * (4 + 2 * ARGS[op]["pages"])
    assert call(op, wsb=need - 1) == WORKSPACE


def test_lists_that_are_empty_or_negative():
    assert call("fork", n=-1) == INVALID and call("release", n=-1) == INVALID
    assert call("fork", P=0) == INVALID
    none = dict(ws=None, wsb=0)
    assert call("fork", n=0, src=None, dst=None, tok=None, cs=None, cd=None, ok=None, **none) == 0
    assert call("release", n=0, req=None, num=None, **none) == 0
    assert call("compact", cap=3) == INVALID  # nine pages may need four moves
    assert kvq.kvq_pages_workspace_size(0, 4) == kvq.kvq_pages_workspace_size(4, 0) == 0
    with pytest.raises(ValueError):
        kvq.pages_workspace(0, 4, device="cpu")


@pytest.mark.parametrize("kw,want", [({"k_pool": None}, INVALID), ({"num_pages": 0}, INVALID), ({"v_pool": 8}, INVALID),
                                     ({"page_size": 8}, UNSUPPORTED), ({"head_dim": 96}, UNSUPPORTED)])
def test_copies_refuse_bad_caches(kw, want):
    L = kvq.load()
    c, b = kvq.CCache(16, 16, 0, 8, 16, 2, 128, 1.0, 1.0), kvq.CBlockCache(16, 16, 16, 8, 16, 2, 128)
    for k, v in kw.items():
        setattr(c, k, v)
        setattr(b, k, v)
    assert L.kvq_copy_pages(ctypes.byref(c), 16, 16, 2, None, None) == want
    assert L.kvq_block_copy_pages(ctypes.byref(b), 16, 16, 2, None, None) == want


def test_copies_refuse_bad_lists():
    L = kvq.load()
    c, b = kvq.CCache(16, 16, 1, 8, 16, 2, 128, 1.0, 1.0), kvq.CBlockCache(16, 16, 16, 8, 16, 2, 128)
    for f, x in ((L.kvq_copy_pages, c), (L.kvq_block_copy_pages, b)):
        assert f(ctypes.byref(x), 16, 16, -1, None, None) == INVALID
        assert f(ctypes.byref(x), None, 16, 2, None, None) == INVALID
        assert f(ctypes.byref(x), 16, None, 2, None, None) == INVALID
        assert f(ctypes.byref(x), None, None, 0, None, None) == 0
    b.scales = 4
    assert L.kvq_block_copy_pages(ctypes.byref(b), 16, 16, 2, None, None) == INVALID


def test_binding_wants_cuda_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    state = kvq.PageState(z, z[:1], z, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvq.kvq_pages_release(state, z, z, None, z, z)
    with pytest.raises(ValueError):
        kvq.kvq_pages_fork(state, z, z, z, z, 16, z, z, z, z)
    with pytest.raises(ValueError):
        kvq.kvq_pages_compact(state, z, z, z, z, z, z)
