"""kvq_block_prefix_attn against the plain 64-bit form of prefix_ref.py, which also gives the
bound of the kernel's error in each value."""
import numpy as np
import pytest
import torch

import block_ref as R
import prefix_ref as X

pytestmark = pytest.mark.gpu

OTHER = 0x4B1D  # a bf16 that rows of nobody hold, before and after


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def cache_of(kvq, s):
    return kvq.BlockKVCache(dev(s.k), dev(s.v), dev(s.scales))


def attend(kvq, s, q, max_q=None, abort=None, sm=None, ws=None, cache=None, groups="own", stream=None, **over):
    N, Hq, D = q.shape
    a = {n: over.get(n, getattr(s, n)) for n in ("tok_start", "lens", "table")}
    out = torch.full((N, Hq, D), OTHER, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = kvq.block_prefix_workspace(N, Hq, s.H, D)
        ws.fill_(0xFF)  # its contents need no preparation
    gs, pp = (s.group_start, s.pre) if isinstance(groups, str) else groups
    kvq.kvq_block_prefix_attn(
        cache or cache_of(kvq, s), q if q.is_cuda else q.cuda(),
        None if a["tok_start"] is None else dev(a["tok_start"]), dev(a["lens"]), dev(a["table"]),
        None if gs is None else dev(gs), None if pp is None else dev(pp), out, ws,
        max_q=max_q or max(1, int(s.n.max())), abort_mask=None if abort is None else dev(abort),
        sm_scale=sm, err_word=err)
    torch.cuda.synchronize()
    return out, int(err.item())


def compare(out, want, tol):
    mine = ~np.isnan(want)
    bits = out.view(torch.int16).cpu().numpy()
    assert (bits[~mine] == OTHER).all(), "rows of nobody were written"
    got = out.float().cpu().numpy().astype(np.float64)
    err = np.abs(got - want) - tol
    err[~mine] = -1
    worst = np.unravel_index(np.nanargmax(err), err.shape)
    ok = not np.isnan(got[mine]).any() and bool(err.max() <= 0)
    assert ok, f"at {worst}: got {got[worst]}, want {want[worst]}, bound {tol[worst]}"


def check(kvq, s, Hq, sm=None, seed=1, skip=(), bits=0, q=None, **kw):
    if q is None:
        q = R.values(np.random.default_rng(seed), s.N, Hq, s.D)
    scale = s.D ** -0.5 if sm is None else sm
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, scale, skip)
    out, err = attend(kvq, s, q[0], sm=sm, **kw)
    assert err == bits
    compare(out, want, tol)
    return out


HEADS = [(1, 1), (1, 4), (2, 2), (4, 4), (8, 4), (8, 8), (3, 6), (5, 3), (9, 1), (2, 7), (1, 16)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", HEADS)
def test_decode_shapes(kvq, H, G, D):
    """One row a request, lengths that end anywhere in a tile and a page, three groups."""
    P = (16, 32, 64)[(H + G) % 3]
    rng = np.random.default_rng([H, G, D])
    s = X.Step(rng, [(128 // P * 2 + 1, [(1, 1), (1, 17), (1, 130)]), (0, [(1, 5), (1, 128)]), (1, [(1, 40)])], H, P, D)
    check(kvq, s, H * G)


@pytest.mark.parametrize("D,P", [(64, 16), (64, 32), (128, 64), (128, 16)])
@pytest.mark.parametrize("H,G,n", [(1, 1, [2, 5]), (2, 4, [1, 2, 0, 3]), (8, 4, [8, 1, 5]), (4, 2, [16, 7, 1]),
                                   (3, 6, [4, 16]), (1, 8, [16, 9]), (2, 3, [40, 1, 33]), (1, 16, [20, 2])])
def test_several_rows(kvq, H, G, n, D, P):
    """Drafted tokens, causal among themselves; rows of a group and of a request that pass a
    block of 128; a request without rows."""
    rng = np.random.default_rng([H, G, D] + n)
    reqs = [(x, max(1, x + int(rng.integers(0, 150)))) for x in n]
    reqs[0] = (n[0], n[0])  # nothing of its own before the step
    s = X.Step(rng, [(3, reqs), (0, [(2, 3)]), (2, reqs[:1])], H, P, D, pad=3)
    check(kvq, s, H * G)
    check(kvq, s, H * G, max_q=max(n) + 13)


@pytest.mark.parametrize("D,P", [(64, 32), (128, 16)])
@pytest.mark.parametrize("H,G,B", [(1, 4, 70), (2, 8, 40), (1, 1, 300)])
def test_many_rows_of_a_group(kvq, H, G, B, D, P):
    """Row blocks of a prefix, the last one part-filled."""
    rng = np.random.default_rng([H, G, B])
    s = X.Step(rng, [(9, [(1, int(rng.integers(1, 30))) for _ in range(B)])], H, P, D)
    check(kvq, s, H * G)


@pytest.mark.parametrize("H,G,D,P", [(8, 4, 128, 16), (8, 8, 128, 64), (2, 4, 64, 32), (1, 5, 128, 32)])
def test_long_and_cut_across_many_ctas(kvq, H, G, D, P):
    rng = np.random.default_rng(2)
    check(kvq, X.Step(rng, [(5000 // P, [(1, 3)])], H, P, D), H * G)
    check(kvq, X.Step(rng, [(4000 // P, [(1, 300), (2, 5)]), (1, [(1, 1500)]), (700 // P, [(1, 1)] * 3)], H, P, D), H * G)
    check(kvq, X.Step(rng, [(0, [(1, 4001)])], H, P, D), H * G)


def test_groups_of_every_kind(kvq):
    """No groups at all (no arrays, empty arrays), requests in front of and behind the groups,
    groups without requests, groups without pages."""
    rng = np.random.default_rng(4)
    s = X.Step(rng, [(0, [(1, 40)]), (4, [(1, 3), (2, 80)]), (0, [(1, 9), (3, 17)])], 2, 16, 64)
    i32 = lambda *x: np.array(x, dtype=np.int32)  # noqa: E731
    first = check(kvq, s, 8)
    for groups in ((None, None), (i32(0), i32()), (i32(1, 3), i32(4)), (i32(0, 0, 1, 1, 3, 3, 3), i32(7, 0, 2, 4, 1, 3)),
                   (i32(1, 2, 3), i32(4, 2)), (i32(5, 5), i32(1)), (i32(0, 5), i32(0))):
        out = check(kvq, s, 8, groups=groups)
        assert float((out.float() - first.float()).abs().max()) < 0.1 * float(first.float().abs().max())


def test_one_row_a_request_without_tok_start(kvq):
    rng = np.random.default_rng(5)
    s = X.Step(rng, [(2, [(1, 7)] * 4)], 2, 32, 128)
    s.tok_start = None
    check(kvq, s, 8)


@pytest.mark.parametrize("D", [64, 128])
def test_scales_far_apart(kvq, D):
    """V scales 2^120 apart, K scales that are no powers of two, both ends of fp32."""
    rng = np.random.default_rng([6, D])
    s = X.Step(rng, [(20, [(1, 33), (3, 200)]), (0, [(1, 150)])], 2, 16, D)
    s.scales[:, :, 0] *= rng.uniform(0.6, 1.4, s.scales.shape[:2]).astype(np.float32)
    s.scales[:, :, 1] = np.exp2(rng.integers(-60, 60, s.scales.shape[:2])).astype(np.float32)
    check(kvq, s, 8)
    s.scales[:, :, 1] = (2.0 ** 100 * rng.uniform(0.6, 1.4, s.scales.shape[:2])).astype(np.float32)
    check(kvq, s, 8)
    s.scales[:, :, 1] = 2.0 ** -120
    check(kvq, s, 8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sm", [0.0, -0.07, 3.0])
def test_score_scales(kvq, D, sm):
    rng = np.random.default_rng([7, D])
    s = X.Step(rng, [(9, [(1, 3), (2, 60)])], 2, 16, D)
    check(kvq, s, 6, sm=sm)


@pytest.mark.parametrize("D", [64, 128])
def test_large_scores_and_a_sink(kvq, D):
    """A first token far above the others whose values are near zero; maxima that grow along the
    sequence by more than the lazy reference allows."""
    rng = np.random.default_rng([8, D])
    s = X.Step(rng, [(24, [(1, 100), (1, 1)])], 1, 16, D)
    q = R.values(rng, s.N, 4, D)
    for t in range(0, 16 * 24, 40):  # later tokens score higher
        s.scales[s.table[0, t // 16], :, 0] = 2.0 ** (-9 + t // 40)
    check(kvq, s, 4, q=q)
    first = s.table[0, 0]
    s.k[first, 0, 0] = np.where(q[1][0, 0] > 0, 0x7E, 0xFE)
    s.v[first, 0, 0] = 0
    check(kvq, s, 4, q=q)


@pytest.mark.parametrize("D", [64, 128])
def test_nan_codes_and_scales_that_nobody_sees(kvq, D):
    """Behind a request's length, and in tokens drafted behind a row: they do not reach it."""
    rng = np.random.default_rng([9, D])
    s = X.Step(rng, [(3, [(5, 12), (1, 20), (4, 131)])], 2, 16, D)
    q = R.values(rng, s.N, 8, D)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5)
    for b in range(s.B):
        last = int(s.lens[b]) - 1
        page, slot = s.table[b, last // 16], last % 16
        s.k[page, :, slot + 1:], s.v[page, :, slot + 1:] = 0x7F, 0xFF
        if s.n[b] > 1:  # the last drafted token: only the last row sees it
            s.v[page, 0, slot, 3], s.k[page, 1, slot, 5] = 0x7F, 0x7F
    out, err = attend(kvq, s, q[0])
    got = out.float().cpu().numpy().astype(np.float64)
    assert err == 0
    for b in range(s.B):
        r = int(s.tok_start[b + 1]) - 1
        if s.n[b] > 1:
            assert np.isnan(got[r, :4, 3]).all() and not np.isnan(np.delete(got[r, :4], 3, axis=1)).any()
            assert np.isnan(got[r, 4:]).all()
            got[r], want[r], tol[r] = 0, 0, 0
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
def test_nan_codes_in_a_prefix_reach_everybody_who_sees_them(kvq, D):
    rng = np.random.default_rng([10, D])
    s = X.Step(rng, [(3, [(1, 12), (2, 20)]), (1, [(1, 4)])], 2, 16, D)
    s.v[s.table[0, 1], 0, 7, 9] = 0x7F
    s.k[s.table[2, 0], 1, 7, 9] = 0xFF
    q = R.values(rng, s.N, 4, D)
    out, err = attend(kvq, s, q[0])
    nan = np.isnan(out.float().cpu().numpy())
    assert err == 0
    want = np.zeros_like(nan)
    want[:3, :2, 9] = True
    want[3, 2:] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("D", [64, 128])
def test_inf_and_nan_queries_stay_in_their_rows(kvq, D):
    rng = np.random.default_rng([11, D])
    s = X.Step(rng, [(10, [(1, 12), (3, 20), (1, 40)])], 2, 16, D)
    q = R.values(rng, s.N, 4, D)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5)
    bad = q[0].clone()
    bad[2, 1, 5], bad[0, 3, 0], bad[4, 0, 1] = float("inf"), float("nan"), float("-inf")
    out, _ = attend(kvq, s, bad)
    got = out.float().cpu().numpy().astype(np.float64)
    for r, h in ((2, 1), (0, 3), (4, 0)):
        assert np.isnan(got[r, h]).all()
        got[r, h], want[r, h] = 0, 0
    assert (np.abs(got - want) <= tol).all()


def test_zero_queries(kvq):
    rng = np.random.default_rng(12)
    s = X.Step(rng, [(10, [(1, 12), (3, 20)])], 2, 16, 128)
    z = torch.zeros(s.N, 8, 128, dtype=torch.bfloat16)
    check(kvq, s, 8, q=(z, z.double().numpy()))


@pytest.mark.parametrize("D", [64, 128])
def test_aborted_requests(kvq, D):
    """The first of a group among them, whose table is not read, and all of another group."""
    rng = np.random.default_rng([13, D])
    s = X.Step(rng, [(5, [(1, 12), (2, 20), (1, 3)]), (2, [(1, 4), (1, 5)])], 2, 16, D, pad=2)
    want_table = s.table.copy()
    abort = np.array([1, 0, 0, 1, 1], dtype=np.uint8)
    q = R.values(rng, s.N, 8, D)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, want_table, D ** -0.5, skip=(0, 3, 4))
    for b in (0, 3, 4):
        s.table[b] = -9
    out, err = attend(kvq, s, q[0], abort=abort)
    assert err == 0
    compare(out, want, tol)


@pytest.mark.parametrize("D", [64, 128])
def test_refused_requests(kvq, D):
    """Bad lengths, more rows than max_q, prefixes that reach into own rows: zeros, and the others
    of the group go on."""
    rng = np.random.default_rng([14, D])
    groups = [(4, [(1, 12), (2, 20), (1, 3)]), (2, [(1, 4), (1, 5)])]
    for b, length, max_q in ((0, 0, None), (1, 64 + 1, None), (2, 16 * 40, None), (0, -1, None), (1, None, 1),
                             (3, 32, None)):
        s = X.Step(rng, groups, 2, 16, D)
        if length is not None:
            s.lens[b] = length
        q = R.values(rng, s.N, 8, D)
        want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5, skip=(b,))
        out, err = attend(kvq, s, q[0], max_q=max_q)
        assert err == kvq.ERRBIT_SEQLEN
        compare(out, want, tol)


@pytest.mark.parametrize("D", [64, 128])
def test_refused_groups(kvq, D):
    rng = np.random.default_rng([15, D])
    s = X.Step(rng, [(4, [(1, 12), (2, 20)]), (2, [(1, 4), (1, 5)])], 2, 16, D, pad=1)
    q = R.values(rng, s.N, 8, D)[0]
    for gs in ([0, 3, 2], [-1, 2, 4], [0, 2, 5], [4, 2, 4], [2 ** 31 - 1, 0, 4]):
        out, err = attend(kvq, s, q, groups=(np.array(gs, dtype=np.int32), s.pre))
        assert err & kvq.ERRBIT_REQ
        assert not out[:s.N - 1].any() and (out[s.N - 1].view(torch.int16) == OTHER).all()
    for pp, skip in (([-1, 2], (0, 1)), ([4, s.MP + 1], (2, 3)), ([2 ** 31 - 1, -2 ** 31], (0, 1, 2, 3))):
        check(kvq, s, 8, groups=(s.group_start, np.array(pp, dtype=np.int32)), skip=skip, bits=kvq.ERRBIT_SEQLEN)


@pytest.mark.parametrize("D", [64, 128])
def test_bad_tok_start(kvq, D):
    rng = np.random.default_rng([16, D])
    s = X.Step(rng, [(4, [(1, 12), (2, 20), (2, 6)])], 2, 16, D, pad=3)
    q = R.values(rng, s.N, 8, D)
    for ts, skip in (([0, 1, 3, 9], ()), ([-1, 1, 3, 5], ()), ([2, 1, 3, 5], (1,)), ([0, 0, 3, 2], (1,))):
        # (rows that do not lie between the ends of their group are refused as well)
        ts = np.array(ts, dtype=np.int32)
        want, tol = X.attend([s.k, s.v], s.scales, q[1], ts, s.lens, s.table, D ** -0.5, skip)
        out, err = attend(kvq, s, q[0], tok_start=ts, max_q=5)
        assert err & kvq.ERRBIT_REQ
        compare(out, want, tol)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_pages_outside_the_pool(kvq, D, bad):
    """In a prefix: the whole group's rows are zeros.  In own tokens: the rows that see them."""
    rng = np.random.default_rng([17, D])
    s = X.Step(rng, [(14, [(1, 12), (2, 300)]), (2, [(3, 36), (1, 5)])], 2, 16, D)
    q = R.values(rng, s.N, 8, D)
    table = s.table.copy()
    table[0, 9] = bad
    out, err = attend(kvq, s, q[0], table=table)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5, skip=(0, 1))
    assert err == kvq.ERRBIT_PAGE
    compare(out, want, tol)
    table = s.table.copy()
    table[2, 4] = bad  # tokens 64 .. 67 of request 2; its rows stand at 65, 66, 67
    out, err = attend(kvq, s, q[0], table=table)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5, skip=(2,))
    assert err == kvq.ERRBIT_PAGE
    compare(out, want, tol)
    s.lens[2] = 2 * 16 + 32 + 1  # rows at 62, 63, 64: only the last one sees it
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5)
    want[int(s.tok_start[3]) - 1], tol[int(s.tok_start[3]) - 1] = 0, 0
    out, err = attend(kvq, s, q[0], table=table)
    assert err == kvq.ERRBIT_PAGE
    compare(out, want, tol)


def test_rows_of_a_wider_projection(kvq):
    rng = np.random.default_rng(18)
    s = X.Step(rng, [(6, [(1, 12), (2, 20)])], 2, 16, 128)
    t, x = R.values(rng, s.N, 12, 128)
    wide = t.cuda()
    q = wide[:, 2:10]
    want, tol = X.attend([s.k, s.v], s.scales, x[:, 2:10], s.tok_start, s.lens, s.table, 128 ** -0.5)
    out, err = attend(kvq, s, q)
    assert err == 0
    compare(out, want, tol)


def test_one_workspace_for_smaller_calls_and_two_streams(kvq):
    """A workspace of more rows serves fewer; calls on two streams with workspaces of their own."""
    rng = np.random.default_rng(19)
    s = X.Step(rng, [(40, [(1, 12)] * 9), (2, [(4, 200)])], 2, 16, 128)
    ws = kvq.block_prefix_workspace(4 * s.N, 8, 2, 128)
    ws.fill_(0xFF)
    q = R.values(rng, s.N, 8, 128)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, 128 ** -0.5)
    out, _ = attend(kvq, s, q[0], ws=ws)
    compare(out, want, tol)
    first = out.clone()
    cache, qd = cache_of(kvq, s), q[0].cuda()
    args = [dev(x) for x in (s.tok_start, s.lens, s.table, s.group_start, s.pre)]
    outs = [torch.zeros_like(first) for _ in range(2)]
    spaces = [kvq.block_prefix_workspace(s.N, 8, 2, 128) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, w, st in zip(outs, spaces, streams):
            kvq.kvq_block_prefix_attn(cache, qd, *args, o, w, max_q=4, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


def test_captured_and_replayed_with_other_lengths(kvq):
    """The schedule is worked out on the device: a graph's lengths, groups and pages may change."""
    rng = np.random.default_rng(20)
    s = X.Step(rng, [(30, [(1, 12), (2, 90)]), (3, [(1, 200), (1, 1)])], 2, 16, 64, extra_pages=2)
    q = R.values(rng, s.N, 8, 64)
    cache, qd = cache_of(kvq, s), q[0].cuda()
    ts, lens, table, gs, pp = (dev(x) for x in (s.tok_start, s.lens, s.table, s.group_start, s.pre))
    out = torch.zeros(s.N, 8, 64, dtype=torch.bfloat16, device="cuda")
    ws = kvq.block_prefix_workspace(s.N, 8, 2, 64)
    call = lambda: kvq.kvq_block_prefix_attn(cache, qd, ts, lens, table, gs, pp, out, ws, max_q=2)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for cut in (0, 7, 0):
        s.lens[2] = 3 * 16 + 200 - 13 * cut
        lens.copy_(dev(s.lens))
        pp.copy_(dev(s.pre if not cut else np.array([17, 0], dtype=np.int32)))
        out.fill_(7.0)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, 64 ** -0.5)
        compare(out, want, tol)


def test_same_bits_every_time(kvq):
    rng = np.random.default_rng(21)
    s = X.Step(rng, [(100, [(1, 12)] * 20 + [(3, 700)]), (2, [(4, 200)])], 8, 16, 128)
    q = R.values(rng, s.N, 32, 128)[0]
    cache = cache_of(kvq, s)
    first, _ = attend(kvq, s, q, cache=cache)
    for _ in range(5):
        assert torch.equal(attend(kvq, s, q, cache=cache)[0], first)


def test_pools_past_four_gigabytes(kvq):
    """Byte offsets of pages that pass 32 bits."""
    rng = np.random.default_rng(22)
    s = X.Step(rng, [(3, [(1, 12), (1, 20)])], 8, 64, 128)
    NP = 70000
    k, v = (torch.zeros(NP, 8, 64, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.ones(NP, 8, 2, device="cuda")
    at = NP - s.NP
    k[at:], v[at:], sc[at:] = dev(s.k), dev(s.v), dev(s.scales)
    q = R.values(rng, s.N, 32, 128)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, 128 ** -0.5)
    out, err = attend(kvq, s, q[0], cache=kvq.BlockKVCache(k, v, sc), table=np.where(s.table < 0, -1, s.table + at).astype(np.int32))
    assert err == 0
    compare(out, want, tol)


def test_near_kvq_block_attn(kvq):
    """The same sequences without groups by kvq_block_attn, whose fp32 result is rounded here."""
    rng = np.random.default_rng(23)
    s = X.Step(rng, [(64, [(1, int(rng.integers(1, 400))) for _ in range(30)])], 8, 16, 128)
    q = R.values(rng, s.N, 32, 128)
    cache = cache_of(kvq, s)
    out, err = attend(kvq, s, q[0], cache=cache)
    want = torch.zeros(s.N, 32, 128, device="cuda")
    kvq.kvq_block_attn(cache, q[0].cuda(), dev(s.tok_start), dev(s.lens), dev(s.table), want,
                       kvq.block_workspace(s.B, 1, 32, 8, 128))
    torch.cuda.synchronize()
    assert err == 0
    # a rounding to bf16 (2^-8 of a value, rms below 2^-9) and to f16 (2^-11 of a weight)
    assert float((out.float() - want).norm() / want.norm()) < 2.0 ** -9


def test_a_run_of_forked_answers(kvq):
    """One prompt appended, forked, its last page copied; then rounds of rotate-and-append, attention
    over the shared prefix, and two answers that end early, against kvq_block_attn."""
    rng = np.random.default_rng(24)
    H, G, P, D, B, MP, NP, prompt = 2, 4, 16, 128, 6, 10, 64, 59
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st = kvq.PageState(torch.arange(NP, dtype=torch.int32, device="cuda"), i32([NP]),
                       torch.zeros(NP, dtype=torch.int32, device="cuda"), torch.full((B, MP), -1, dtype=torch.int32, device="cuda"),
                       torch.zeros(B, MP, dtype=torch.int32, device="cuda"))
    shares, ws = torch.zeros(NP, dtype=torch.int32, device="cuda"), kvq.pages_workspace(NP, B)
    err = i32([0])
    cache = kvq.BlockKVCache(torch.zeros(NP, H, P, D, dtype=torch.uint8, device="cuda"),
                             torch.zeros(NP, H, P, D, dtype=torch.uint8, device="cuda"), torch.ones(NP, H, 2, device="cuda"))
    inv, m = kvq.kvq_rope_inv_freq(D)
    rope = kvq.Rope(inv.cuda(), kvq.ROPE_HALF, m)
    ok1, ok = torch.zeros(1, dtype=torch.uint8, device="cuda"), torch.zeros(B - 1, dtype=torch.uint8, device="cuda")
    kvq.kvq_pages_update(st, acq_req=i32([0]), acq_first=i32([0]), acq_npages=i32([4]), acq_ok=ok1, err_word=err)
    k, v = R.values(rng, prompt, H, D)[0].cuda(), R.values(rng, prompt, H, D)[0].cuda()
    lens = i32([prompt] + [0] * (B - 1))
    kvq.kvq_rope_block_append(cache, rope, None, None, k, v, i32([0] + [prompt] * B), lens, st.block_table, err_word=err)
    cs, cd = i32([0] * (B - 1)), i32([0] * (B - 1))
    kvq.kvq_pages_fork(st, shares, i32([0] * (B - 1)), i32(list(range(1, B))), i32([prompt] * (B - 1)), P, cs, cd, ok, ws, err_word=err)
    kvq.kvq_block_copy_pages(cache, cs, cd, err_word=err)
    lens.fill_(prompt)
    gs, pp = i32([0, B]), i32([prompt // P])
    aws, bws = kvq.block_prefix_workspace(2 * B, H * G, H, D), kvq.block_workspace(B, 2, H * G, H, D)
    live = np.ones(B, dtype=int)
    for step in range(12):
        n = 1 + (step % 3 == 1)
        counts = n * live
        ts = i32([0] + np.cumsum(counts).tolist())
        N = int(counts.sum())
        lens += i32(counts.tolist())
        need = [b for b in range(B) if live[b] and -(-int(lens[b]) // P) > -(-(int(lens[b]) - n) // P)]
        if need:
            first = [-(-(int(lens[b]) - n) // P) for b in need]
            kvq.kvq_pages_update(st, acq_req=i32(need), acq_first=i32(first), acq_npages=i32([1] * len(need)),
                                 acq_ok=torch.zeros(len(need), dtype=torch.uint8, device="cuda"), err_word=err)
        q = R.values(rng, N, H * G, D)[0].cuda()
        q2 = torch.empty_like(q)
        kvq.kvq_rope_block_append(cache, rope, q, q2, R.values(rng, N, H, D)[0].cuda(), R.values(rng, N, H, D)[0].cuda(),
                                  ts, lens, st.block_table, err_word=err)
        mask = torch.zeros(B, dtype=torch.uint8, device="cuda")
        kvq.kvq_check_tags(st.block_table, lens, P, st.page_tags, st.expected_tags, mask)
        out, want = torch.zeros(N, H * G, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, H * G, D, device="cuda")
        kvq.kvq_block_prefix_attn(cache, q2, ts, lens, st.block_table, gs, pp, out, aws, max_q=2, abort_mask=mask, err_word=err)
        kvq.kvq_block_attn(cache, q2, ts, lens, st.block_table, want, bws, max_q=2, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and not mask.any()
        assert float((out.float() - want).norm() / want.norm()) < 2.0 ** -9
        if step == 5:  # two answers end; the first of the group is one of them
            gone = [0, 3]
            pages = [-(-int(lens[b]) // P) for b in gone]
            kvq.kvq_pages_release(st, shares, i32(gone), None, i32(pages), ws, err_word=err)
            live[gone] = 0
            lens[gone[0]] = lens[gone[1]] = 0
    left = [b for b in range(B) if live[b]]
    kvq.kvq_pages_release(st, shares, i32(left), None, i32([-(-int(lens[b]) // P) for b in left]), ws, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and int(st.free_count.item()) == NP and not shares.any()


def shared(s, G):
    """Both of the kernels that attend to own tokens: a row a request, and more than they take at once."""
    return ({}, {"max_q": 16 // G + 1})


@pytest.mark.parametrize("D", [64, 128])
def test_largest_value_scales(kvq, D):
    """Up to the largest fp32, with codes so small that the values are finite."""
    rng = np.random.default_rng([24, D])
    s = X.Step(rng, [(9, [(1, 200), (1, 3), (1, 90)]), (0, [(1, 640)])], 2, 16, D)
    s.v &= 0x87  # at most 7 2^-9
    e = rng.integers(124, 128, s.scales.shape[:2])
    s.scales[:, :, 1] = np.ldexp(rng.integers(4, 8, e.shape) / 4.0, e)
    s.scales[::3, :, 1] = np.float32(2.0 ** 127)
    s.scales[1::5, :, 1] = np.finfo(np.float32).max
    for kw in shared(s, 4):
        check(kvq, s, 8, **kw)


@pytest.mark.parametrize("D", [64, 128])
def test_smallest_value_scales(kvq, D):
    """Values near fp32's smallest normal number; scales that are subnormal.  An output may also be off
    by a step of a subnormal bf16, 2^-133."""
    rng = np.random.default_rng([25, D])
    s = X.Step(rng, [(9, [(1, 200), (1, 3)]), (0, [(1, 300)])], 2, 16, D)
    s.v = (s.v & 0x87) | 0x70  # 128 .. 240
    s.scales[:, :, 1] = 2.0 ** -126
    s.scales[1::2, :, 1] = np.float32(2.0 ** -126 * 0.8125)
    s.scales[2::5, :, 1] = np.float32(2.0 ** -149)
    q = R.values(rng, s.N, 8, D)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5)
    for kw in shared(s, 4):
        out, err = attend(kvq, s, q[0], **kw)
        assert err == 0
        compare(out, want, tol - 1e-37 + 2.0 ** -133)


def scored(rng, scores, pages, reqs, D, scale):
    """A step of one group whose token j scores scores[j] ln 2 (at score scale ln 2) for every row: q and K are
    zeros but in one dim, so that a score is one exact product."""
    s = X.Step(rng, [(pages, reqs)], 1, 16, D)
    s.k[:] = 0
    s.scales[:, :, 0] = 1.0
    s.scales[:, :, 1] = scale
    codes = R.encode(scores / 16.0)
    assert (R.decode(codes) * 16.0 == scores).all()
    for b in range(s.B):
        at = np.arange(int(s.lens[b]))
        s.k[s.table[b, at // 16], 0, at % 16, 5] = codes[at]
    q = np.zeros((s.N, 4, D))
    q[:, :, 5] = 16.0
    return s, R.bf16(q), (R.bf16(q).float().numpy().astype(np.float64))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e,jump", [(0, 56.0), (60, 56.0), (110, 56.0), (110, 112.0), (-60, 224.0)])
def test_large_values_behind_a_growing_maximum(kvq, D, e, jump):
    """Scores that grow by 2^56 and more within a row, in the prefix and in own tokens: the references
    are undone without overflow, whatever the V scales."""
    rng = np.random.default_rng([26, D, abs(e)])
    scores = rng.choice([0.4375, 0.8125, 2.75], 1000)
    scores[300], scores[700] = jump, jump + (8 if jump < 112 else 16)
    s, q, x = scored(rng, scores, 600 // 16, [(1, 408 - 8), (1, 30), (1, 300)], D, 2.0 ** e)
    s.v = (s.v & 0x87) | 0x30  # 0.5 .. 0.94
    for kw in shared(s, 4):
        check(kvq, s, 4, q=(q, x), sm=float(np.log(2.0)), **kw)


@pytest.mark.parametrize("gap", [16, 18, 20, 22, 24])
def test_tokens_below_a_sink_without_value(kvq, gap):
    """The first token's score is some `gap` ln 2 above the others', its values are zero: the others'
    weights, all alike, are the output."""
    rng = np.random.default_rng([27, gap])
    scores = np.full(2000, {16: 0.4375, 18: 0.5625, 20: 0.625, 22: 0.8125, 24: 0.875}[gap])
    scores[0] = gap
    s, q, x = scored(rng, scores, 100, [(1, 300), (1, 9)], 128, 1.0)
    s.v = (s.v & 0x07) | 0x38  # 1 .. 1.875, one sign: equal roundings do not even out
    s.v[s.table[0, 0], :, 0] = 0
    for kw in shared(s, 4):
        check(kvq, s, 4, q=(q, x), sm=float(np.log(2.0)), **kw)


@pytest.mark.parametrize("D", [64, 128])
def test_long_sums_of_one_sign(kvq, D):
    """Every weight alike and every value positive, so that what the tensor cores' additions lose adds up;
    requests enough that one CTA sums whole prefixes."""
    rng = np.random.default_rng([28, D])
    s = X.Step(rng, [(40000 // 64, [(1, 20), (1, 1)])], 1, 64, D)
    s.v &= 0x7F
    q = np.zeros((s.N, 4, D))
    check(kvq, s, 4, q=(R.bf16(q), q))
    B = 160  # groups of one, the same pages: 160 rows of work for as many CTAs or fewer
    s.B = s.N = B
    s.n, s.lens = np.ones(B, dtype=np.int32), np.full(B, s.lens[1], dtype=np.int32)
    s.table = np.repeat(s.table[1:], B, 0)
    s.tok_start = s.group_start = np.arange(B + 1, dtype=np.int32)
    s.pre = np.full(B, s.pre[0], dtype=np.int32)
    one, tol = X.attend([s.k, s.v], s.scales, q[:1], s.tok_start[:2], s.lens[:1], s.table[:1], D ** -0.5)
    q = np.zeros((B, 4, D))
    out, err = attend(kvq, s, R.bf16(q))
    assert err == 0
    compare(out, np.repeat(one, B, 0), np.repeat(tol, B, 0))


def test_the_largest_max_q_and_its_workspace(kvq):
    """max_q is a limit, not a size; a workspace that is too small, or not aligned, is refused."""
    rng = np.random.default_rng(29)
    s = X.Step(rng, [(3, [(1, 20), (6, 9)])], 2, 16, 64)
    check(kvq, s, 4, max_q=2 ** 31 - 1)
    q = R.values(rng, s.N, 4, 64)[0]
    ws = kvq.block_prefix_workspace(s.N, 4, 2, 64)
    for bad in (ws[:-1], ws[16:]):
        with pytest.raises(kvq.KvqError):
            attend(kvq, s, q, ws=bad)


def test_binding_refuses_other_shapes(kvq):
    rng = np.random.default_rng(31)
    s = X.Step(rng, [(3, [(1, 20), (1, 9)])], 2, 16, 64)
    q = R.values(rng, s.N, 4, 64)[0]
    one = np.array([1], dtype=np.int32)
    for groups in ((None, s.pre), (s.group_start, None), (s.group_start, s.pre[:0]), (s.group_start.astype(np.int64), s.pre)):
        with pytest.raises(ValueError):
            attend(kvq, s, q, groups=groups)
    with pytest.raises(ValueError):
        attend(kvq, s, q, abort=np.zeros(3, dtype=np.uint8))
    with pytest.raises(ValueError):
        attend(kvq, s, q.float())
    with pytest.raises(ValueError):
        attend(kvq, s, q, lens=one)


def test_many_groups_of_one(kvq):
    """More groups than the plan takes at once, a request each, and empty ones in between."""
    rng = np.random.default_rng(30)
    s = X.Step(rng, [(1, [(1, int(rng.integers(1, 40)))]) if g % 3 else (2, []) for g in range(1700)], 1, 16, 64)
    check(kvq, s, 4)


@pytest.mark.parametrize("max_q", [1, 9])
def test_nobody_takes_part(kvq, max_q):
    """Every request aborted, or without rows, or refused: zeros, and rows of nobody left as they were."""
    rng = np.random.default_rng(32)
    s = X.Step(rng, [(3, [(1, 20), (1, 9)]), (1, [(1, 30)])], 2, 16, 128, pad=2)
    check(kvq, s, 8, max_q=max_q, skip=(0, 1, 2), abort=np.ones(3, dtype=np.uint8))
    lens = s.lens.copy()
    s.lens[:] = [0, -1, 1 << 30]
    check(kvq, s, 8, max_q=max_q, skip=(0, 1, 2), bits=2)  # KVQ_ERRBIT_SEQLEN
    s.lens = lens
    s.tok_start[:] = 0
    check(kvq, s, 8, max_q=max_q)
    s.tok_start[:] = [0, 0, 0, s.N]  # one request has all the rows
    check(kvq, s, 8, max_q=9)
