"""The block-scaled cache's operators at the edges of what include/kvq.h promises."""
import numpy as np
import pytest
import torch

import block_ref as R
from test_gpu_block_cache import assert_cache, dev, run_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,P,D", [(3, 32, 64), (1, 64, 128), (1, 32, 64)])
def test_append_prompts_with_short_tails(kvq, H, P, D):
    """Few kv heads and several pages a CTA, full ones and short tails in turn: the maxima
    that the warps of a full page exchange are its own."""
    rng = np.random.default_rng([H, P, D, 31])
    n = rng.integers(1, 3, 900) * P + rng.integers(1, 17, 900)
    s = R.Step(rng, n, n, H, P, D)
    mag = np.exp2(rng.integers(-12, 13, (s.N, H, 1)))
    kt, vt = (R.bf16(rng.standard_normal((s.N, H, D)) * mag) for _ in range(2))
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kt.double().numpy(), vt.double().numpy()], s.tok_start, s.lens, s.table)
    c, err = run_append(kvq, s, (kt, vt))
    assert err == 0
    assert_cache(c, pools, scales)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attend(kvq, s, q, max_q, table=None, ws=None, sm=None, abort=None):
    Hq, D = q.shape[1:]
    out = torch.full((q.shape[0], Hq, D), -77.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = kvq.block_workspace(s.B, max_q, Hq, s.H, D)
    kvq.kvq_block_attn(kvq.BlockKVCache(dev(s.k), dev(s.v), dev(s.scales)), q.cuda(), dev(s.tok_start),
                       dev(s.lens), dev(s.table if table is None else table), out, ws, max_q=max_q,
                       abort_mask=None if abort is None else dev(abort), sm_scale=sm, err_word=err)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64), int(err.item())


def compare(got, want, tol):
    err = np.abs(got - want) - tol
    worst = np.unravel_index(np.nanargmax(err), err.shape)
    assert not np.isnan(got).any() and err.max() <= 0, \
        f"at {worst}: got {got[worst]}, want {want[worst]}, bound {tol[worst]}"


@pytest.mark.parametrize("D,max_q", [(64, 1), (64, 6), (128, 1), (128, 3), (128, 6)])
def test_largest_value_scales(kvq, D, max_q):
    """V scales up to the largest fp32, with codes so small that the values are finite: block_ref's
    bound, in which nothing depends on a scale's size."""
    rng = np.random.default_rng([D, max_q, 32])
    s = R.Step(rng, [1, max_q, 1], [200, 90, 640], 2, 16, D)
    s.v &= 0x87  # at most 7 2^-9
    e = rng.integers(124, 128, s.scales.shape[:2])
    s.scales[:, :, 1] = np.ldexp(rng.integers(4, 8, e.shape) / 4.0, e)
    s.scales[::3, :, 1] = np.float32(2.0 ** 127)
    s.scales[1::5, :, 1] = np.finfo(np.float32).max
    q, qx = R.values(rng, s.N, 8, D)
    want, tol = R.attend([s.k, s.v], s.scales, qx, s.tok_start, s.lens, s.table, D ** -0.5, max_q=max_q)
    got, err = attend(kvq, s, q, max_q)
    assert err == 0
    compare(got, want, tol)


MANY = 320  # requests over the same pages: more than CTAs, so that one sums whole rows


def one_dim(s, scores, Hq):
    """Makes score j of every row scores[j] * ln 2, at score scale ln 2: q and K are 0 but in one dim,
    so that a score is one exact product.  Copies the first request MANY times; returns q."""
    s.k[:] = 0
    codes = R.encode(scores / 16.0)
    assert (R.decode(codes) * 16.0 == scores).all()
    s.scales[:, :, 0] = 1.0
    at = np.arange(len(scores))
    s.k[s.table[0][at // s.P], :, at % s.P, 5] = codes[:, None]
    s.B = s.N = MANY
    s.n, s.lens = np.ones(MANY, dtype=np.int32), np.full(MANY, len(scores), dtype=np.int32)
    s.tok_start, s.table = np.arange(MANY + 1, dtype=np.int32), np.repeat(s.table, MANY, 0)
    q = np.zeros((MANY, Hq, s.D))
    q[:, :, 5] = 16.0
    return R.bf16(q)


def exact(s, scores, G, magnitude=False):
    """Softmax of 2^scores times the values (or their magnitudes): [heads, D]."""
    v = R.gather(s.v & 0x7F if magnitude else s.v, s.scales, 1, s.table[0], np.arange(len(scores)))
    w = np.exp2(scores - scores.max())
    return np.repeat(np.einsum("j,jhd->hd", w, v) / w.sum(), G, 0)


def roundings(top, L):
    """Relative error of weights and sums where scores are exact products of at most `top` ln 2: a
    score's factor is rounded three times, 3 2^-24; a weight's exponential and pieces leave 2^-21 and
    2^-18; sums add (L / 16 + 64) 2^-24; all of it twice, for the denominator."""
    return 2 * (top * np.log(2) * 3 * 2.0 ** -24 * 2 + 2.0 ** -21 + 2.0 ** -18 + (L / 16 + 64) * 2.0 ** -24)


@pytest.mark.parametrize("D,max_q", [(64, 1), (128, 1), (128, 6)])
@pytest.mark.parametrize("L", [40, 3000])
@pytest.mark.parametrize("top", [2.75, 11.0])
def test_smallest_value_scales(kvq, D, max_q, L, top):
    """Values near fp32's smallest normal number, in blocks whose scales are subnormal or the
    library's smallest, 2^-126, among them a token with a larger score (or none) whose block's
    scale is smaller still.  An output may also be off by 2^-149, fp32's smallest step."""
    rng = np.random.default_rng([D, max_q, L, 33])
    G = 4
    s = R.Step(rng, [1], [L], 1, 16, D)
    scores = rng.choice([0.4375, 0.8125, 2.75], L)
    scores[3] = top
    q = one_dim(s, scores, G)
    s.v = (s.v & 0x87) | 0x70  # 128 .. 240
    s.v[s.table[0, 0]] = 0
    s.scales[:, :, 1] = 2.0 ** -126
    s.scales[s.table[0, 1::2], :, 1] = np.float32(2.0 ** -126 * 0.8125)
    s.scales[s.table[0, 0], :, 1] = np.float32(2.0 ** -149)
    got, err = attend(kvq, s, q, max_q, sm=float(np.log(2.0)))
    assert err == 0
    tol = roundings(11, L) * exact(s, scores, G, True) + 2.0 ** -149
    compare(got, np.broadcast_to(exact(s, scores, G), got.shape), np.broadcast_to(tol, got.shape))


@pytest.mark.parametrize("D,max_q", [(64, 1), (128, 1), (128, 6)])
@pytest.mark.parametrize("e", [60, 90, 110])
def test_large_values_behind_a_growing_maximum(kvq, D, max_q, e):
    """Scores that grow by 2^56 within a row whose V scales are 2^e: the factor that undoes the
    references is applied without overflow."""
    rng = np.random.default_rng([D, max_q, e, 34])
    L, G = 700, 4
    s = R.Step(rng, [1], [L], 1, 16, D)
    scores = rng.choice([0.4375, 0.8125, 2.75], L)
    scores[300] = 56.0
    q = one_dim(s, scores, G)
    s.v = (s.v & 0x87) | 0x30  # 0.5 .. 0.94
    s.scales[:, :, 1] = 2.0 ** e
    got, err = attend(kvq, s, q, max_q, sm=float(np.log(2.0)))
    assert err == 0
    tol = roundings(56, L) * exact(s, scores, G, True)
    compare(got, np.broadcast_to(exact(s, scores, G), got.shape), np.broadcast_to(tol, got.shape))


@pytest.mark.parametrize("L,max_q", [(300, 1), (300, 6), (9000, 1), (9000, 6)])
@pytest.mark.parametrize("gap", [16, 18, 20, 22, 24])
def test_tokens_below_a_sink_without_value(kvq, gap, L, max_q):
    """The first token's score is about gap ln 2 above the others', its values are zero: the others'
    weights are the output.  include/kvq.h: a weight is held to 2^-30 of the row's largest (times
    their V scales, here equal), that is to 2^(gap - 30) of itself, beside its own roundings."""
    rng = np.random.default_rng([gap, L, max_q, 35])
    G, D = 4, 128
    s = R.Step(rng, [1], [L], 1, 16, D)
    scores = np.full(L, {16: 0.4375, 18: 0.5625, 20: 0.625, 22: 0.8125, 24: 0.875}[gap])  # fractions: weights of all bits
    scores[0] = gap
    q = one_dim(s, scores, G)
    s.v = (s.v & 0x07) | 0x38  # 1 .. 1.875, one sign: equal roundings do not even out
    s.v[s.table[0, 0], :, 0] = 0
    s.scales[:, :, 1] = 1.0
    got, err = attend(kvq, s, q, max_q, sm=float(np.log(2.0)))
    assert err == 0
    want = exact(s, scores, G)
    tol = (2.0 ** (gap - scores[1] - 30) + roundings(gap, L)) * want
    compare(got, np.broadcast_to(want, got.shape), np.broadcast_to(tol, got.shape))


SIZES = [(8, 4, 128), (8, 1, 128), (8, 8, 128), (5, 4, 64), (7, 2, 64), (5, 3, 128), (1, 5, 128), (3, 6, 64)]


@pytest.mark.parametrize("H,G,D", SIZES)
def test_a_workspace_serves_fewer_rows_and_requests(kvq, H, G, D):
    """Sized for max_q rows of B requests it serves every smaller max_q, over narrow and wide tables."""
    size = [kvq.kvq_block_attn_workspace_size(4, n, H * G, H, D) for n in range(1, 150)]
    assert all(a <= b for a, b in zip(size, size[1:]))
    assert all(kvq.kvq_block_attn_workspace_size(b, 9, H * G, H, D) <= size[8] for b in range(5))
    most = 40
    ws = kvq.block_workspace(4, most, H * G, H, D)
    rng = np.random.default_rng([H, G, D, 36])
    for n in (1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 40):
        s = R.Step(rng, [n, 1], [n + 30, 50], H, 16, D)
        q, _ = R.values(rng, s.N, H * G, D)
        for table in (s.table, np.pad(s.table, ((0, 0), (0, 256)), constant_values=-1)):
            got, err = attend(kvq, s, q, n, table=table, ws=ws)
            own, _ = attend(kvq, s, q, n, table=table)
            assert err == 0 and np.array_equal(got, own)


@pytest.mark.parametrize("H,G,D,max_q", [(2, 4, 64, 8), (2, 1, 64, 70), (2, 1, 128, 8), (8, 4, 128, 8),
                                         (1, 4, 128, 70), (1, 16, 64, 20)])
@pytest.mark.parametrize("before", [9, 3001])
def test_bad_page_zeroes_only_the_rows_that_see_it(kvq, H, G, D, max_q, before):
    """Rows that end before the first token of a page outside the pool are as ever; stale NaN codes
    of other requests do not reach them."""
    rng = np.random.default_rng([H, G, D, before, 37])
    n = [max_q, 2, max_q, max_q]
    lens = [before + max_q, 40, before + max_q, 13 + max_q]
    s = R.Step(rng, n, lens, H, 16, D)
    q, _ = R.values(rng, s.N, H * G, D)
    base, err = attend(kvq, s, q, max_q)
    assert err == 0
    s.v[s.table[1, 0]] = s.v[s.table[3, 0]] = 0x7F  # requests 1 and 3 read NaN
    table, dead = s.table.copy(), np.zeros(s.N, dtype=bool)
    last = (lens[0] - 1) // 16
    for b, lp in ((0, last), (2, max(last - 1, 0))):
        table[b, lp] = (-1, s.NP)[b == 2]
        row = np.arange(s.tok_start[b], s.tok_start[b + 1])
        dead[row] = lens[b] - n[b] + 1 + np.arange(n[b]) > lp * 16
    got, err = attend(kvq, s, q, max_q, table=table)
    assert err == kvq.ERRBIT_PAGE
    mine = np.r_[s.tok_start[0]:s.tok_start[1], s.tok_start[2]:s.tok_start[3]]
    assert dead[mine].any() and not dead[mine].all()
    assert (got[dead] == 0).all()
    keep = mine[~dead[mine]]
    assert np.array_equal(got[keep], base[keep])
    assert np.isnan(got[s.tok_start[1]:s.tok_start[2]]).all()


def test_an_input_without_its_output_is_refused(kvq):
    c = kvq.BlockKVCache.empty(4, 2, 16, 64)
    rope = kvq.Rope(torch.ones(32, dtype=torch.float64, device="cuda"))
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.ones(1, dtype=torch.int32, device="cuda")
    t = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for q, q_out in ((x, None), (None, x)):
        with pytest.raises(ValueError):
            kvq.kvq_rope_block_append(c, rope, q, q_out, x, x, None, i, t)
        with pytest.raises(ValueError):
            kvq.kvq_rope(rope, i, x, x, q, q_out)
        if q is not None:
            with pytest.raises(ValueError):
                kvq.kvq_rope(rope, i, q, q_out)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def append_f32(pools, scales, new, tok_start, lens, table):
    """R.append with the fp32 products that include/kvq.h states for scales of the caller's own."""
    P, f = pools[0].shape[2], np.float32
    for b in range(len(lens)):
        row, n = int(tok_start[b]), int(tok_start[b + 1] - tok_start[b])
        p0 = int(lens[b]) - n
        for lp in range(p0 // P, (p0 + n - 1) // P + 1) if n else ():
            page = int(table[b, lp])
            lo, hi = max(p0, lp * P), min(p0 + n, lp * P + P)
            old = lo - lp * P
            for i in range(2):
                x = new[i][row + lo - p0:row + hi - p0]
                for h in range(pools[0].shape[1]):
                    s = f(R.block_scale(float(np.abs(x[:, h]).max())))
                    if old:
                        was = f(scales[page, h, i])
                        s = max(s, was)
                        if s > was:
                            pools[i][page, h, :old] = R.encode(
                                R.decode(pools[i][page, h, :old]).astype(f) * (was / s))
                    scales[page, h, i] = s
                    pools[i][page, h, old:hi - lp * P] = R.encode(x[:, h].astype(f) * (f(1) / s))


@pytest.mark.parametrize("H,P,D,n", [(2, 16, 128, 3), (3, 32, 64, 9), (1, 64, 128, 400), (8, 16, 64, 300),
                                     (3, 32, 128, 200)])
def test_append_to_blocks_with_scales_of_the_callers(kvq, H, P, D, n):
    """Blocks whose old scales are no powers of two, ties of x / s and neighbours of ties among the
    values, by all kernels (short, staged and wide)."""
    rng = np.random.default_rng([H, P, D, n, 38])
    B = 60
    before = rng.integers(1, 2 * P, B)
    s = R.Step(rng, [n] * B, before + n, H, P, D)
    s.scales[:] = np.exp2(rng.integers(-9, 3, s.scales.shape)) * rng.choice(
        [1.0, 1.25, 1.75, 1.75, 5 / 3, 1.9999999, rng.uniform(1, 2)], s.scales.shape)
    s.scales[::7] = np.float32(3e38)
    s.scales[3::11] = np.float32(2.0 ** -130 * 1.3)
    kt, vt = (R.bf16(rng.integers(-255, 256, (s.N, H, D)) * np.exp2(rng.integers(-10, -4, (s.N, H, 1))))
              for _ in range(2))
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    append_f32(pools, scales, [kt.double().numpy(), vt.double().numpy()], s.tok_start, s.lens, s.table)
    c, err = run_append(kvq, s, (kt, vt))
    assert err == 0
    assert_cache(c, pools, scales)


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("H,P,D,B,n", [(2, 16, 128, 300, 290), (3, 32, 64, 900, 880), (8, 64, 128, 200, 150)])
def test_append_part_of_a_prompt_among_idle_slots(kvq, H, P, D, B, n, rope):
    """Fixed slots, most of them without rows, one with a part of a prompt: no more rows than slots."""
    rng = np.random.default_rng([H, P, D, B, 39])
    rows = np.zeros(B, dtype=np.int64)
    rows[[3, B // 2, B - 1]] = 1, n, 2
    s = R.Step(rng, rows, np.where(rows > 0, rows + rng.integers(0, 50, B), 0), H, P, D)
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    if rope:
        from test_gpu_block_cache import check_rope_append
        return check_rope_append(kvq, s, rng, 4 * H, D, True)
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    lens, table = s.lens.copy(), s.table.copy()
    table[B // 2, 1] = s.NP
    R.append(pools, scales, [kx, vx], s.tok_start, lens, table)
    c, err = run_append(kvq, s, (kt, vt), table=table)
    assert err == kvq.ERRBIT_PAGE
    assert_cache(c, pools, scales)


@pytest.mark.parametrize("Hq", [1, 3, 8, 11])
@pytest.mark.parametrize("H,P,D", [(8, 16, 128), (9, 16, 64), (2, 64, 128)])
def test_rope_append_prompts_with_any_number_of_query_heads(kvq, H, P, D, Hq):
    """Fewer query heads than a staged group of heads holds, and no multiple of it."""
    from test_gpu_block_cache import check_rope_append, prompts
    rng = np.random.default_rng([H, P, D, Hq, 40])
    check_rope_append(kvq, prompts(rng, H, P, D), rng, Hq, D // 2, Hq % 2 == 0)


def test_idle_slots_in_a_captured_step(kvq):
    """A captured append of fixed slots, replayed while rows move from many requests to one and
    back, on a stream of its own."""
    H, P, D, B = 2, 16, 64, 80
    rng = np.random.default_rng(41)
    s = R.Step(rng, [0] * B, [200] * B, H, P, D)
    c = kvq.BlockKVCache(dev(s.k), dev(s.v), dev(s.scales))
    N = B
    k, v = (torch.zeros(N, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ts, lens = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (B + 1, B))
    table, err = dev(s.table), torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvq.kvq_block_append(c, k, v, ts, lens, table, err_word=err)
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    length = rng.integers(0, 50, B)
    for n in ([1] * B, [0] * 7 + [80] + [0] * 72, [0] * B, [0, 2] * 40, [35] + [0] * 78 + [45], [1] * B):
        n = np.array(n)
        start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        (kt, kx), (vt, vx) = R.values(rng, N, H, D), R.values(rng, N, H, D)
        length += n
        k.copy_(kt.cuda()), v.copy_(vt.cuda()), ts.copy_(dev(start))
        lens.copy_(dev(length.astype(np.int32)))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        R.append(pools, scales, [kx, vx], start, length, s.table)
        assert int(err.item()) == 0
        assert_cache(c, pools, scales)
