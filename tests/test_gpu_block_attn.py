"""kvq_block_attn against the plain 64-bit form of block_ref.py, which also
gives the bound of the kernel's error in each value."""
import numpy as np
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def cache_of(kvq, s):
    return kvq.BlockKVCache(dev(s.k), dev(s.v), dev(s.scales))


def attend(kvq, s, q, max_q, tok_start="own", lens=None, table=None, abort=None, cache=None,
           sm=None, ws=None):
    Hq, D = q.shape[1:]
    out = torch.full((q.shape[0], Hq, D), -77.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = kvq.block_workspace(s.B, max_q, Hq, s.H, D)
        ws.fill_(0xFF)  # its contents need no preparation
    ts = s.tok_start if isinstance(tok_start, str) else tok_start
    kvq.kvq_block_attn(cache or cache_of(kvq, s), q if q.is_cuda else q.cuda(),
                       None if ts is None else dev(ts), dev(s.lens if lens is None else lens),
                       dev(s.table if table is None else table), out, ws, max_q=max_q,
                       abort_mask=None if abort is None else dev(abort), sm_scale=sm, err_word=err)
    torch.cuda.synchronize()
    return out.cpu().numpy(), int(err.item())


def compare(got, want, tol):
    mine = ~np.isnan(want)
    assert (got[~mine] == -77.0).all(), "rows of nobody were written"
    err = np.abs(got.astype(np.float64) - want) - tol
    err[~mine] = -1
    worst = np.unravel_index(np.nanargmax(err), err.shape)
    ok = not np.isnan(got[mine]).any() and bool(err.max() <= 0)
    assert ok, f"at {worst}: got {got[worst]}, want {want[worst]}, bound {tol[worst]}"


def check(kvq, s, Hq, max_q=None, rng=None, **kw):
    rng = rng or np.random.default_rng(1)
    q, qx = R.values(rng, s.N, Hq, s.D)
    sm = s.D ** -0.5
    max_q = max_q or max(1, int(s.n.max()))
    want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, s.table, sm, max_q=max_q)
    got, err = attend(kvq, s, q, max_q, **kw)
    assert err == 0
    compare(got, want, tol)
    if s.D == 128 and 8 < max_q * (Hq // s.H) <= 16 and s.MP * s.P < 4096:
        # and by the kernel that such calls take where requests can be long
        table = wide(s)
        want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, table, sm, max_q=max_q)
        wide_got, err = attend(kvq, s, q, max_q, table=table, **kw)
        assert err == 0
        compare(wide_got, want, tol)
    return got


def wide(s):
    """The step's block table with room for 4,096 tokens."""
    more = -(-4096 // s.P) - s.MP
    return np.pad(s.table, ((0, 0), (0, max(0, more))), constant_values=-1)


HEADS = [(1, 1), (1, 4), (2, 2), (4, 4), (8, 4), (8, 8), (3, 6), (5, 3), (9, 1), (2, 7), (1, 16)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", HEADS)
def test_decode_shapes(kvq, H, G, D):
    """One row a request; lengths that end anywhere in a tile and a page."""
    P = (16, 32, 64)[(H + G) % 3]
    rng = np.random.default_rng([H, G, D])
    s = R.Step(rng, [1] * 7, [1, 2, 15, 16, 17, 100, 333], H, P, D)
    check(kvq, s, H * G)


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
@pytest.mark.parametrize("H,G,n", [(1, 1, [2, 5]), (2, 4, [1, 2, 0, 3]), (8, 4, [8, 1, 5]), (4, 2, [16, 7, 1]),
                                   (3, 6, [4, 16]), (1, 8, [16, 9]), (8, 8, [3, 16]), (2, 3, [40, 1, 33]),
                                   (1, 16, [20, 2])])
def test_several_rows(kvq, H, G, n, D, P):
    """Drafted tokens: causal among themselves, row tiles of 4, 8 and 16, several
    tiles and several row blocks."""
    rng = np.random.default_rng([H, G, D] + n)
    lens = [x + int(rng.integers(0, 150)) for x in n]
    lens[0] = n[0]  # nothing before the step
    s = R.Step(rng, n, lens, H, P, D, pad=3)
    check(kvq, s, H * G)
    check(kvq, s, H * G, max_q=max(n) + 13)  # a larger promise, another tiling


@pytest.mark.parametrize("H,G,D,P", [(8, 4, 128, 16), (8, 8, 128, 64), (2, 4, 64, 32), (1, 5, 128, 32)])
def test_long_and_cut_across_many_ctas(kvq, H, G, D, P):
    """One long request (many parts a row) and a ragged batch with short ones."""
    rng = np.random.default_rng(2)
    check(kvq, R.Step(rng, [2], [9001], H, P, D), H * G)
    check(kvq, R.Step(rng, [1, 1, 1, 1, 1, 1], [3000, 1, 40, 5000, 17, 800], H, P, D), H * G)


@pytest.mark.parametrize("H,G,n,P", [(8, 4, 8, 16), (2, 8, 4, 64), (3, 5, 3, 32), (1, 12, 9, 16)])
def test_drafts_over_long_and_short_contexts(kvq, H, G, n, P):
    """Several rows over contexts that end anywhere in a 128-token tile, cut across
    CTAs and not, in one and in several row blocks."""
    rng = np.random.default_rng([H, G, n])
    lens = [n, 127, 128, 129, 255 + n, 1000, 5003, 2 * n]
    check(kvq, R.Step(rng, [n, 1, n, n - 1, 2, n, n, n], lens, H, P, 128, pad=1), H * G)
    check(kvq, R.Step(rng, [n], [3000 + n], H, P, 128), H * G)


@pytest.mark.parametrize("H,G,n,L,D", [(8, 4, 1, 2600, 128), (1, 4, 8, 9100, 128), (2, 8, 1, 5000, 128),
                                       (8, 1, 1, 2100, 64), (1, 4, 2, 9300, 64), (2, 5, 2, 5000, 128)])
def test_long_sums_do_not_drift(kvq, H, G, n, L, D):
    """Values of one sign, over so many requests that a CTA sums thousands of tokens of
    each.  All requests share one prefix."""
    rng = np.random.default_rng([H, G, n, L])
    s = R.Step(rng, [n], [L], H, 16, D)
    s.v &= 0x7F
    s.v[(s.v & 0x7F) == 0x7F] = 0x7E
    s.k[:] = rng.integers(0x20, 0x30, s.k.shape, dtype=np.uint8) | (s.k & 0x80)
    B, few = 160, 6
    q, qx = R.values(rng, B * n, H * G, D)
    ts, lens = (np.arange(B + 1) * n).astype(np.int32), np.full(B, L, dtype=np.int32)
    s.B = B
    got, err = attend(kvq, s, q, n, tok_start=ts, lens=lens, table=np.repeat(s.table, B, 0))
    assert err == 0
    rows = few * n
    want, tol = R.attend([s.k, s.v], s.scales, qx[:rows], ts[:few + 1], lens[:few],
                         np.repeat(s.table, few, 0), D ** -0.5, max_q=n)
    compare(got[:rows], want, tol)
    # no drift: roundings even out, and at most 64 additions in a row truncate, each
    # half of 2^-23 on average: 64 2^-24 = 3.8e-6
    rel = (got[:rows] - want) / want
    assert abs(rel.mean()) < 4e-6
    bad = np.repeat(s.table, B, 0)
    bad[1, 3], bad[2, -1] = -1, s.NP  # a bad page near a row's start and at its end
    again, err = attend(kvq, s, q, n, tok_start=ts, lens=lens, table=bad)
    assert err == kvq.ERRBIT_PAGE
    assert (again[n:3 * n] == 0).all()
    keep = np.r_[0:n, 3 * n:B * n]
    assert np.array_equal(again[keep], got[keep])


@pytest.mark.parametrize("n,L", [(8, 9100), (1, 9100)])
def test_long_contexts_with_scales_far_apart(kvq, n, L):
    """Scales that grow and shrink by 2^60 over thousands of tokens of one CTA: the
    references move before and after long sums leave the tensor core."""
    rng = np.random.default_rng([n, L])
    s = R.Step(rng, [n], [L], 1, 16, 128)
    pages = s.table[0, :-(-L // 16)]
    at = np.arange(len(pages))
    s.scales[pages, 0, 1] = np.exp2(np.round(30 * np.sin(at / 90.0) + rng.integers(-3, 4, len(at))))
    s.scales[pages, 0, 0] = np.exp2(rng.integers(-9, -6, len(at)))
    B, few = 160, 4
    q, qx = R.values(rng, B * n, 4, 128)
    ts, lens = (np.arange(B + 1) * n).astype(np.int32), np.full(B, L, dtype=np.int32)
    s.B = B
    got, err = attend(kvq, s, q, n, tok_start=ts, lens=lens, table=np.repeat(s.table, B, 0))
    assert err == 0
    want, tol = R.attend([s.k, s.v], s.scales, qx[:few * n], ts[:few + 1], lens[:few],
                         np.repeat(s.table, few, 0), 128 ** -0.5, max_q=n)
    compare(got[:few * n], want, tol)


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 16), (1, 3, 64, 32), (3, 1, 128, 64)])
def test_prompt_parts_among_decode_rows(kvq, H, G, D, P):
    """Many row blocks of one request beside single rows."""
    rng = np.random.default_rng([H, G, D])
    n = [1] * 9 + [150] + [1, 3, 0, 1] + [70]
    s = R.Step(rng, n, np.add(n, rng.integers(0, 400, len(n))), H, P, D, pad=2)
    check(kvq, s, H * G)


def test_many_drafts(kvq):
    rng = np.random.default_rng(14)
    n = rng.integers(0, 5, 700)
    s = R.Step(rng, n, np.where(n > 0, n + rng.integers(0, 300, 700), 0), 2, 32, 128)
    check(kvq, s, 8, max_q=4)


def test_many_requests(kvq):
    """More requests than CTAs and than a CTA's threads, some without rows."""
    rng = np.random.default_rng(3)
    n = rng.integers(0, 3, 900)
    s = R.Step(rng, n, np.where(n > 0, n + rng.integers(0, 40, 900), 0), 2, 16, 64)
    check(kvq, s, 4, max_q=2)


@pytest.mark.parametrize("max_q", [1, 6])
def test_scales_far_apart(kvq, max_q):
    """Pages whose V scales differ by 2^120, and not powers of two: a block of
    large values with little softmax weight beside one of small values."""
    rng = np.random.default_rng(4)
    s = R.Step(rng, [1, max_q, 1], [200, 90, 640], 2, 16, 128)
    s.scales[:, :, 0] *= rng.uniform(0.6, 1.9, s.scales.shape[:2]).astype(np.float32)
    s.scales[:, :, 1] = np.exp2(rng.integers(-60, 60, s.scales.shape[:2])) * \
        rng.uniform(0.6, 1.9, s.scales.shape[:2])
    check(kvq, s, 8)


@pytest.mark.parametrize("D", [64, 128])
def test_zero_blocks_keep_their_weight(kvq, D):
    """V blocks of zeros carry the smallest scale, 2^-126: their tokens count in
    the denominator all the same."""
    rng = np.random.default_rng(5)
    s = R.Step(rng, [1, 4], [100, 64], 1, 16, D)
    for lp in (0, 2, 3):
        for b in range(2):
            s.v[s.table[b, lp]] = 0
            s.scales[s.table[b, lp], :, 1] = 2.0 ** -126
    s.k[:] = 0x10  # equal keys: every token weighs the same
    check(kvq, s, 3)


def test_large_scores(kvq):
    """Scores of several hundreds, and q of very different sizes."""
    rng = np.random.default_rng(6)
    s = R.Step(rng, [1, 2, 1], [300, 77, 20], 2, 16, 128)
    q, _ = R.values(rng, s.N, 8, 128)
    q[0] *= 64
    q[1] *= 2.0 ** -40
    q[2] = 0
    qx = q.double().numpy()
    for max_q in (2, 5):
        want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, s.table, 0.25, max_q=max_q)
        got, err = attend(kvq, s, q, max_q, sm=0.25)
        assert err == 0
        compare(got, want, tol)


@pytest.mark.parametrize("sm", [0.0, -0.05])
def test_zero_and_negative_score_scale(kvq, sm):
    rng = np.random.default_rng(15)
    s = R.Step(rng, [2, 1, 3], [150, 33, 300], 2, 16, 128)
    q, qx = R.values(rng, s.N, 8, 128)
    for max_q in (3, 5):
        want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, s.table, sm, max_q=max_q)
        got, err = attend(kvq, s, q, max_q, sm=sm)
        assert err == 0
        compare(got, want, tol)


def test_infinite_and_nan_queries_stay_in_their_rows(kvq):
    """A row of q with an inf or a NaN is NaN; the rows beside it are as ever."""
    rng = np.random.default_rng(16)
    s = R.Step(rng, [3, 2], [90, 40], 2, 16, 128)
    q, qx = R.values(rng, s.N, 8, 128)
    for max_q in (3, 5):
        base, _ = attend(kvq, s, q, max_q)
        bad = q.clone()
        bad[1, 2, 7], bad[3, 5, 100] = float("inf"), float("nan")
        got, err = attend(kvq, s, bad, max_q)
        assert err == 0
        hit = np.zeros((s.N, 8), dtype=bool)
        hit[1, 2] = hit[3, 5] = True
        assert np.isnan(got[hit]).all() and np.array_equal(got[~hit], base[~hit])


def test_two_graphs_share_a_workspace(kvq):
    """Graphs of calls of different sizes replayed in turn over one workspace."""
    rng = np.random.default_rng(17)
    steps = [R.Step(rng, [4, 1, 2], [700, 5, 90], 2, 16, 128), R.Step(rng, [1] * 9, [300] * 9, 2, 16, 128),
             R.Step(rng, [8, 8], [5000, 64], 2, 16, 128)]
    ws = torch.empty(max(kvq.kvq_block_attn_workspace_size(s.B, int(s.n.max()), 8, 2, 128) for s in steps),
                     dtype=torch.uint8, device="cuda")
    runs = []
    for s in steps:
        q, _ = R.values(rng, s.N, 8, 128)
        n = int(s.n.max())
        want, _ = attend(kvq, s, q, n)
        args = (cache_of(kvq, s), q.cuda(), dev(s.tok_start), dev(s.lens), dev(s.table),
                torch.zeros(s.N, 8, 128, device="cuda"), ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kvq.kvq_block_attn(*args, max_q=n)
        runs.append((graph, args, want))
    for k in (0, 1, 2, 1, 0, 2):
        graph, args, want = runs[k]
        args[5].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(args[5].cpu().numpy(), want)


def test_nan_codes_stay_where_they_are_not_seen(kvq):
    """NaN codes behind a request's end, in unused pages and in drafted tokens
    that earlier rows do not see; a row that sees one is NaN."""
    rng = np.random.default_rng(7)
    for H, G, n, D in ((2, 4, [4, 1, 6], 128), (1, 2, [2, 1, 5], 64), (8, 4, [8, 1, 3], 128),
                       (2, 1, [3, 1, 6], 128), (1, 16, [5, 1, 7], 128)):
        s = R.Step(rng, n, [37, 21, 50], H, 16, D)
        q, qx = R.values(rng, s.N, H * G, D)
        want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, s.table, D ** -0.5,
                             max_q=max(n))
        for b in range(3):  # slots past the end
            L = int(s.lens[b])
            page = s.table[b, (L - 1) // 16]
            s.k[page, :, (L - 1) % 16 + 1:] = 0xFF
            s.v[page, :, (L - 1) % 16 + 1:] = 0x7F
        free = sorted(set(range(s.NP)) - set(s.table.ravel().tolist()))
        s.k[free], s.v[free] = 0x7F, 0x7F
        got, err = attend(kvq, s, q, max(n))
        assert err == 0
        compare(got, want, tol)
        # the last token of requests 0 and 2 is NaN: only their last rows see it
        for b in (0, 2):
            L = int(s.lens[b])
            s.v[s.table[b, (L - 1) // 16], :, (L - 1) % 16] = 0x7F
            s.k[s.table[b, (L - 1) // 16], 0, (L - 1) % 16, 3] = 0xFF
        got, err = attend(kvq, s, q, max(n))
        last = [int(s.tok_start[1]) - 1, int(s.tok_start[3]) - 1]
        assert np.isnan(got[last]).all()
        keep = np.ones(s.N, dtype=bool)
        keep[last] = False
        compare(got[keep], want[keep], tol[keep])


@pytest.mark.parametrize("extra", [1, 250])
def test_aborted_and_bad_requests(kvq, extra):
    """Aborted rows are zeros and their pages are not read; bad lengths, too many
    rows and bad pages zero theirs; bad starts leave theirs; others as ever."""
    rng = np.random.default_rng(8)
    n = [2, 1, 3, 1, 2, 5, 1]
    s = R.Step(rng, n, [40, 33, 60, 20, 70, 25, 90], 2, 16, 128, extra_pages=extra, pad=2)
    q, qx = R.values(rng, s.N, 8, 128)
    want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, s.table, 128 ** -0.5,
                         skip=(1, 2, 3, 4, 5), max_q=4)
    abort = np.zeros(7, dtype=np.uint8)
    abort[1] = 1
    lens, table = s.lens.copy(), s.table.copy()
    table[1, 0] = 10 ** 6           # aborted: not even looked at
    lens[2] = 2                     # below its three rows
    lens[3] = s.MP * 16 + 1
    table[4, 1] = -1
    got, err = attend(kvq, s, q, 4, lens=lens, table=table, abort=abort)  # request 5: five rows
    assert err == kvq.ERRBIT_SEQLEN | kvq.ERRBIT_PAGE
    compare(got, want, tol)
    ts = s.tok_start.copy()
    ts[3], ts[4] = ts[4] + 1, ts[3]  # requests 2 .. 4 overlap or run backwards
    got, err = attend(kvq, s, q, 5, tok_start=ts)
    assert err & kvq.ERRBIT_REQ
    base, _ = attend(kvq, s, q, 5)
    same = [*range(int(ts[2])), *range(int(ts[6]), int(ts[7]))]
    assert np.array_equal(got[same], base[same])


@pytest.mark.parametrize("max_q", [1, 6])
def test_bad_page_of_a_row_cut_across_ctas(kvq, max_q):
    rng = np.random.default_rng(9)
    s = R.Step(rng, [1, 1], [4000, 4000], 8, 16, 128)
    q, qx = R.values(rng, s.N, 32, 128)
    base, _ = attend(kvq, s, q, max_q)
    table = s.table.copy()
    table[0, 100] = s.NP
    got, err = attend(kvq, s, q, max_q, table=table)
    assert err == kvq.ERRBIT_PAGE
    assert (got[0] == 0).all() and np.array_equal(got[1], base[1])


@pytest.mark.parametrize("max_q", [1, 7])
def test_repeatable_and_page_order(kvq, max_q):
    """The same bits every time, wherever the pages lie, and without starts."""
    rng = np.random.default_rng(10)
    s = R.Step(rng, [1] * 5, [1000, 3, 500, 77, 2048], 2, 32, 128)
    q, _ = R.values(rng, 5, 8, 128)
    a, _ = attend(kvq, s, q, max_q)
    b, _ = attend(kvq, s, q, max_q, tok_start=None)
    perm = rng.permutation(s.NP)
    t = R.Step(rng, [1] * 5, s.lens, 2, 32, 128)
    t.k, t.v, t.scales = np.empty_like(s.k), np.empty_like(s.v), np.empty_like(s.scales)
    t.k[perm], t.v[perm], t.scales[perm] = s.k, s.v, s.scales
    t.table = np.where(s.table >= 0, perm[np.maximum(s.table, 0)], -1).astype(np.int32)
    c, _ = attend(kvq, t, q, max_q)
    assert np.array_equal(a, b) and np.array_equal(a, c)


@pytest.mark.parametrize("max_q", [3, 5])
def test_strided_q_side_stream_and_graph(kvq, max_q):
    rng = np.random.default_rng(11)
    s = R.Step(rng, [3, 1, 2], [70, 5, 300], 2, 16, 128)
    wide, x = R.values(rng, s.N, 12, 128)
    want, tol = R.attend([s.k, s.v], s.scales, x[:, 2:10], s.tok_start, s.lens, s.table, 128 ** -0.5,
                         max_q=max_q)
    w = wide.cuda()
    got, _ = attend(kvq, s, w[:, 2:10], max_q)
    compare(got, want, tol)
    c, ts, lens, table = cache_of(kvq, s), dev(s.tok_start), dev(s.lens), dev(s.table)
    ws = [kvq.block_workspace(3, max_q, 8, 2, 128) for _ in range(2)]
    outs = [torch.zeros(s.N, 8, 128, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):  # two calls at once, each with its workspace
        for o, k, st in zip(outs, ws, streams):
            kvq.kvq_block_attn(c, w[:, 2:10], ts, lens, table, o, k, max_q=max_q, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(o.cpu().numpy(), got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_block_attn(c, w[:, 2:10], ts, lens, table, outs[0], ws[0], max_q=max_q)
    outs[0].zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(outs[0].cpu().numpy(), got)


def test_offsets_past_32_bits(kvq):
    """A pool of over 4 GB: the last pages' codes and scales are the ones read and
    written."""
    H, P, D = 8, 64, 128
    NP = (1 << 32) // (H * P * D) + 40
    rng = np.random.default_rng(12)
    s = R.Step(rng, [1, 2], [130, 70], H, P, D)
    kp, vp = (torch.zeros(NP, H, P, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = torch.ones(NP, H, 2, device="cuda")
    off = NP - s.NP
    kp[off:], vp[off:], scales[off:] = dev(s.k), dev(s.v), dev(s.scales)
    c = kvq.BlockKVCache(kp, vp, scales)
    far = np.where(s.table >= 0, s.table + off, -1).astype(np.int32)
    q, qx = R.values(rng, s.N, 16, D)
    for max_q in (2, 9):
        want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, s.table, D ** -0.5, max_q=max_q)
        got, err = attend(kvq, s, q, max_q, table=far, cache=c)
        assert err == 0
        compare(got, want, tol)
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    kvq.kvq_block_append(c, kt.cuda(), vt.cuda(), dev(s.tok_start), dev(s.lens), dev(far))
    pools, sc = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, sc, [kx, vx], s.tok_start, s.lens, s.table)
    assert np.array_equal(kp[off:].cpu().numpy(), pools[0])
    assert np.array_equal(vp[off:].cpu().numpy(), pools[1])
    assert np.array_equal(scales[off:].cpu().numpy(), sc) and not kp[:off].any()


def test_a_run_of_the_operators_together(kvq):
    """A prompt and then draft steps as a server makes them: rotate, quantise and
    append, attend, all captured in one graph; the drafted tokens that are
    turned down are overwritten by the next step.  Against the same steps in 64
    bits from the cache's own codes, and the prefix read back at the end."""
    H, G, P, D, B, T = 2, 4, 16, 128, 3, 3
    rng = np.random.default_rng(13)
    prompts = np.array([40, 7, 19])
    s = R.Step(rng, prompts, prompts + 40, H, P, D)
    c = cache_of(kvq, s)
    f, m = kvq.kvq_rope_inv_freq(D, scaling=kvq.ROPE_RAMP, factor=4.0, orig_len=64.0)
    rope = kvq.Rope(f.cuda(), kvq.ROPE_HALF, m)
    table, err = dev(s.table), torch.zeros(1, dtype=torch.int32, device="cuda")
    (kt, kx), (vt, _) = R.values(rng, int(prompts.sum()), H, D), R.values(rng, int(prompts.sum()), H, D)
    kvq.kvq_rope_block_append(c, rope, None, None, kt.cuda(), vt.cuda(), dev(s.tok_start),
                              dev(prompts.astype(np.int32)), table, err_word=err)
    N = B * T + 2  # padded
    qkv = torch.zeros(N, (G + 2) * H, D, dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :G * H], qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]
    qr, out = torch.zeros(N, G * H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, G * H, D, device="cuda")
    ts, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B + 1, B))
    ws = kvq.block_workspace(B, T, G * H, H, D)

    def step():
        kvq.kvq_rope_block_append(c, rope, q, qr, k, v, ts, lens, table, err_word=err)
        kvq.kvq_block_attn(c, qr, ts, lens, table, out, ws, max_q=T, err_word=err)

    step()  # no rows yet: library set-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    length = prompts.copy()
    for t in range(8):
        n = rng.integers(1, T + 1, B)
        start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        x, xx = R.values(rng, N, (G + 2) * H, D)
        qkv.copy_(x.cuda())
        ts.copy_(dev(start))
        lens.copy_(dev((length + n).astype(np.int32)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        pools, scales = [c.k_pool.cpu().numpy(), c.v_pool.cpu().numpy()], c.scales.cpu().numpy()
        want, tol = R.attend(pools, scales, qr.double().cpu().numpy(), start, length + n, s.table, D ** -0.5,
                             max_q=T)
        rows = int(start[-1])
        err_ = np.abs(out.cpu().numpy()[:rows] - want[:rows]) - tol[:rows]
        assert err_.max() <= 0, t
        # the step's own tokens lie in the cache: within half an e4m3 step of their block's scale
        for b in range(B):
            at = np.arange(length[b], length[b] + n[b])
            xv = xx[start[b]:start[b + 1], (G + 1) * H:]
            got = R.gather(pools[1], scales, 1, s.table[b], at)
            sc = scales[s.table[b][at // P]][:, :, 1][:, :, None]
            assert (np.abs(got - xv) <= 2.0 ** -4 * np.abs(xv) + 2.0 ** -10 * sc).all()
        length += rng.integers(1, n + 1)  # the accepted ones
    back = torch.zeros(int(length.sum()), H, D, dtype=torch.bfloat16, device="cuda")
    back_v = torch.zeros_like(back)
    st = np.concatenate([[0], np.cumsum(length)]).astype(np.int32)
    kvq.kvq_block_read(c, dev(st), None, table, back, back_v, err_word=err)
    assert int(err.item()) == 0
    pools, scales = [c.k_pool.cpu().numpy(), c.v_pool.cpu().numpy()], c.scales.cpu().numpy()
    for b in range(B):
        assert np.array_equal(back[st[b]:st[b + 1]].double().cpu().numpy(),
                              R.gather(pools[0], scales, 0, s.table[b], np.arange(length[b])))
