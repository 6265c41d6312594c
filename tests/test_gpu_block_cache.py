"""The block-scaled cache's writing and reading (kvq_rope, kvq_block_append,
kvq_rope_block_append, kvq_block_read) against the plain 64-bit forms of
block_ref.py: codes and scales bit for bit where nothing is rotated."""
import numpy as np
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

# bf16 rounds by at most half a step, 2^-8 of the value; sines and products in
# fp32 are off by a few 2^-24 of the pair, the frequency table (2^-53, times a
# position below 2^31) by 2^-21 radians
BF16_HALF, ROT = 2.0 ** -8, 2.0 ** -19


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def cache_of(kvq, s):
    return kvq.BlockKVCache(dev(s.k), dev(s.v), dev(s.scales))


def assert_cache(c, pools, scales, what=""):
    got = c.scales.cpu().numpy()
    assert np.array_equal(got.view(np.uint32), scales.view(np.uint32)), f"{what}: scales differ"
    for name, t, want in (("k", c.k_pool, pools[0]), ("v", c.v_pool, pools[1])):
        g = t.cpu().numpy()
        assert np.array_equal(g, want), \
            f"{what}: {int((g != want).sum())} codes of {name} differ, first at " \
            f"{tuple(int(x[0]) for x in np.nonzero(g != want))}"


def inv_freq(rd, base=10000.0):
    return base ** (-2.0 * np.arange(rd // 2) / rd)


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------

def check_rotation(got, x, pos, f, half, m=1.0):
    want = R.rotate(x, pos, f, half, m)
    pair = np.abs(x).copy()
    rd = 2 * len(f)
    if half:
        pair[..., :rd] += np.abs(np.concatenate([x[..., rd // 2:rd], x[..., :rd // 2]], -1))
    else:
        pair[..., :rd] += np.abs(x[..., :rd].reshape(*x.shape[:-1], -1, 2)[..., ::-1]
                                 .reshape(*x.shape[:-1], rd))
    g = got.double().cpu().numpy()
    err = np.abs(g - want) - (BF16_HALF * np.abs(want) + ROT * abs(m) * pair)
    assert err.max() <= 0, np.unravel_index(err.argmax(), err.shape)
    assert np.array_equal(g[..., rd:], x[..., rd:])


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("D,rd", [(128, 128), (128, 64), (128, 16), (128, 96), (64, 64), (64, 48)])
@pytest.mark.parametrize("N,Hq,Hk", [(1, 1, 0), (7, 5, 1), (33, 40, 8), (5, 72, 8)])
def test_rope(kvq, half, D, rd, N, Hq, Hk):
    rng = np.random.default_rng([D, rd, N, Hq])
    q, qx = R.values(rng, N, Hq, D)
    k, kx = R.values(rng, N, max(Hk, 1), D)
    pos = rng.integers(0, 100000, N).astype(np.int32)
    f = inv_freq(rd)
    rope = kvq.Rope(dev(f), kvq.ROPE_HALF if half else kvq.ROPE_INTERLEAVED, 1.25)
    qo, ko = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
    if Hk:
        kvq.kvq_rope(rope, dev(pos), q.cuda(), qo, k.cuda(), ko)
        check_rotation(ko, kx, pos, f, half, 1.25)
    else:
        kvq.kvq_rope(rope, dev(pos), q.cuda(), qo)
    check_rotation(qo, qx, pos, f, half, 1.25)


@pytest.mark.parametrize("half", [True, False])
def test_rope_far_and_negative_positions(kvq, half):
    """Positions up to the ends of int32: the angle is reduced without loss."""
    pos = np.array([0, 1, 2, 1 << 20, (1 << 24) + 1, 1 << 30, 2 ** 31 - 1, -1, -7, -2 ** 31],
                   dtype=np.int32)
    rng = np.random.default_rng(3)
    q, qx = R.values(rng, len(pos), 3, 128)
    f = inv_freq(128)
    out = torch.empty_like(q).cuda()
    kvq.kvq_rope(kvq.Rope(dev(f), kvq.ROPE_HALF if half else kvq.ROPE_INTERLEAVED), dev(pos),
                 q.cuda(), out)
    check_rotation(out, qx, pos, f, half)


def test_rope_in_place_strided_and_non_finite(kvq):
    """q and k as slices of one projection, rotated in place; v beside them and
    rows of other tokens stay; inf and NaN stay within their pair."""
    rng = np.random.default_rng(4)
    N, Hq, Hk, D, rd = 9, 6, 2, 64, 32
    qkv, x = R.values(rng, N, Hq + 2 * Hk, D)
    qkv[2, 1, 3] = float("inf")
    qkv[3, 0, 40] = float("nan")  # not rotated
    x = qkv.double().numpy()
    t = qkv.cuda()
    q, k = t[:, :Hq], t[:, Hq:Hq + Hk]
    f = inv_freq(rd)
    pos = np.arange(N, dtype=np.int32) + 5
    kvq.kvq_rope(kvq.Rope(dev(f), kvq.ROPE_INTERLEAVED), dev(pos), q, q, k, k)
    got = t.double().cpu().numpy()
    assert np.array_equal(got[:, Hq + Hk:], x[:, Hq + Hk:])
    assert np.isnan(got[3, 0, 40]) and np.isnan(got[3, 0]).sum() == 1
    odd = np.zeros_like(got, dtype=bool)
    odd[2, 1, 2:4] = odd[3, 0, 40] = True
    assert np.isfinite(got[~odd]).all() and not np.isfinite(got[2, 1, 2:4]).any()
    clean = np.where(odd, 0.0, x)
    want = R.rotate(clean[:, :Hq + Hk], pos, f, False)
    err = np.abs(np.where(odd, want_like(want, got), got)[:, :Hq + Hk] - want)
    assert (err <= BF16_HALF * np.abs(want) + ROT * 8).all()


def want_like(want, got):
    full = np.zeros_like(got)
    full[:, :want.shape[1]] = want
    return full


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def run_append(kvq, s, new, tok_start="own", lens=None, table=None, cache=None, strided=False):
    c = cache or cache_of(kvq, s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = new
    if strided:
        both = torch.cat([k, v], 1).cuda()
        k, v = both[:, :s.H], both[:, s.H:]
    ts = s.tok_start if isinstance(tok_start, str) else tok_start
    kvq.kvq_block_append(c, k.cuda(), v.cuda(), None if ts is None else dev(ts),
                         dev(s.lens if lens is None else lens),
                         dev(s.table if table is None else table), err_word=err)
    torch.cuda.synchronize()
    return c, int(err.item())


SHAPES = [(1, 16, 64), (2, 16, 128), (3, 32, 128), (8, 16, 128), (8, 64, 128), (5, 64, 64), (2, 32, 64)]


@pytest.mark.parametrize("H,P,D", SHAPES)
@pytest.mark.parametrize("n,before", [
    ([1], [0]), ([1, 1, 1, 1], [0, 15, 16, 63]), ([3, 1, 0, 8, 2], [5, 64, 9, 60, 0]),
    ([200, 1, 65, 17], [0, 7, 30, 16])])
def test_append_matches_bit_for_bit(kvq, H, P, D, n, before):
    """Ragged steps into new, half full and several pages: codes, scales and
    everything that is not written."""
    rng = np.random.default_rng([H, P, D, len(n)])
    s = R.Step(rng, n, np.add(n, before), H, P, D)
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kx, vx], s.tok_start, s.lens, s.table)
    c, err = run_append(kvq, s, (kt, vt), strided=len(n) == 4)
    assert err == 0
    assert_cache(c, pools, scales)
    run_append(kvq, s, (kt, vt), cache=c)  # the same rows again change nothing
    assert_cache(c, pools, scales, "again")


@pytest.mark.parametrize("H,P,D", [(2, 16, 128), (4, 64, 128), (3, 32, 64)])
def test_append_token_by_token_with_growing_values(kvq, H, P, D):
    """Decode steps whose values grow and shrink: scales grow by steps of one and
    of many powers of two, old codes are requantised, down to zero."""
    rng = np.random.default_rng(5)
    B, steps = 3, P + 5
    s = R.Step(rng, [1] * B, [steps] * B, H, P, D)
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    c = cache_of(kvq, s)
    for t in range(steps):
        mag = 2.0 ** rng.integers(-30, 30, (B, H, 1)) if t % 3 else 1.5 ** t
        kt, vt = R.bf16(rng.standard_normal((B, H, D)) * mag), R.bf16(rng.standard_normal((B, H, D)) * mag)
        lens = np.full(B, t + 1, dtype=np.int32)
        R.append(pools, scales, [kt.double().numpy(), vt.double().numpy()], None, lens, s.table)
        run_append(kvq, s, (kt, vt), tok_start=None, lens=lens, cache=c)
    assert_cache(c, pools, scales)


def test_append_special_values(kvq):
    """Zeros, amax exactly 448 2^k, inf, NaN, subnormals, the largest bf16."""
    H, P, D = 2, 16, 128
    rng = np.random.default_rng(6)
    rows = []
    for top in (0.0, 448.0, 450.0, 1.75, float("inf"), float("nan"), 1e-39, 3.38e38, -448 * 2.0 ** -20):
        x = rng.standard_normal((H, D)) * (min(abs(top), 1e30) if np.isfinite(top) and top else 0.0) * 2e-3
        x[:, 7] = top
        rows.append(x)
    kt = R.bf16(np.array(rows))
    vt = R.bf16(-np.array(rows))
    B = len(rows)
    s = R.Step(rng, [1] * B, [1] * B, H, P, D)
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kt.double().numpy(), vt.double().numpy()], None, s.lens, s.table)
    c, err = run_append(kvq, s, (kt, vt), tok_start=None)
    assert err == 0
    assert_cache(c, pools, scales)


def test_append_leaves_bad_requests_and_pages_out(kvq):
    H, P, D = 2, 16, 64
    rng = np.random.default_rng(7)
    n = [2, 3, 20, 1, 4]
    s = R.Step(rng, n, [10, 3, 25, 40, 9], H, P, D, extra_pages=1, pad=6)
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    table = s.table.copy()
    table[2, 1] = s.NP      # half of request 2's rows
    table[3, 2] = -5
    lens = s.lens.copy()
    lens[1] = 2             # below its three rows
    lens[4] = s.MP * P + 1  # over the table
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kx, vx], s.tok_start, lens, table)
    c, err = run_append(kvq, s, (kt, vt), lens=lens, table=table)
    assert err == kvq.ERRBIT_SEQLEN | kvq.ERRBIT_PAGE
    assert_cache(c, pools, scales)
    # starts that run backwards, below zero or past the rows
    for bad in ([0, 2, 1, 25, 26, 30], [-1, 2, 5, 25, 26, 30], [0, 2, 5, 25, 26, s.N + 1]):
        ts = np.array(bad, dtype=np.int32)
        pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
        R.append(pools, scales, [kx, vx], ts, np.maximum(s.lens, 24), table_all(s))
        c, err = run_append(kvq, s, (kt, vt), tok_start=ts, lens=np.maximum(s.lens, 24),
                            table=table_all(s))
        assert err & kvq.ERRBIT_REQ
        assert_cache(c, pools, scales, bad)


def table_all(s):
    """A table whose rows are all distinct pages where the pool has them, else -1."""
    t = np.full((s.B, s.MP), -1, dtype=np.int32)
    flat = np.arange(min(s.NP, t.size), dtype=np.int32)
    t.reshape(-1)[:len(flat)] = flat
    return t


def test_append_many_requests_and_long_prompt(kvq):
    """More requests than the CTAs have threads, one of them a long prompt."""
    H, P, D = 1, 32, 64
    rng = np.random.default_rng(8)
    n = rng.integers(0, 3, 700)
    n[333] = 1500
    before = rng.integers(0, 40, 700)
    s = R.Step(rng, n, n + before, H, P, D)
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kx, vx], s.tok_start, s.lens, s.table)
    c, err = run_append(kvq, s, (kt, vt))
    assert err == 0
    assert_cache(c, pools, scales)


# Prompts large enough for the staged kernel (heads times page size of 128 and
# more) and for the one without staging: ragged, starting in the middle of pages,
# with odd head counts, the last page of a prompt short.
PROMPTS = [(8, 16, 128), (9, 16, 64), (2, 64, 128), (5, 32, 128), (3, 64, 64),  # staged
           (1, 16, 128), (3, 32, 64), (1, 64, 128)]


def prompts(rng, H, P, D, pad=5):
    n = np.array([130 * P, 1, 9 * P + 3, 0, 200 * P + 7, P, 3])
    return R.Step(rng, n, n + np.array([0, 5, 11, 3, 2 * P + 1, 0, P - 1]), H, P, D, pad=pad)


@pytest.mark.parametrize("H,P,D", PROMPTS)
def test_append_prompts(kvq, H, P, D):
    rng = np.random.default_rng([H, P, D, 5])
    s = prompts(rng, H, P, D)
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kx, vx], s.tok_start, s.lens, s.table)
    c, err = run_append(kvq, s, (kt, vt), strided=True)
    assert err == 0
    assert_cache(c, pools, scales)


def mixed(rng, H, P, D):
    """Rows of decode and draft steps with parts of two prompts among them."""
    n = np.array([1] * 30 + [9 * P + 3] + [2, 0, 5] * 5 + [1] * 25 + [4 * P, 1])
    return R.Step(rng, n, n + rng.integers(0, 70, len(n)), H, P, D, pad=3)


@pytest.mark.parametrize("H,P,D", [(8, 16, 128), (3, 32, 64), (1, 64, 128)])
def test_append_prompt_parts_among_decode_rows(kvq, H, P, D):
    rng = np.random.default_rng([H, P, D, 6])
    s = mixed(rng, H, P, D)
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    table, lens = s.table.copy(), s.lens.copy()
    table[30, (lens[30] - 1) // P - 1] = -1  # a bad page late in the first prompt's part
    lens[0] = -5
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kx, vx], s.tok_start, lens, table)
    c, err = run_append(kvq, s, (kt, vt), lens=lens, table=table)
    assert err == kvq.ERRBIT_SEQLEN | kvq.ERRBIT_PAGE
    assert_cache(c, pools, scales)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("H,P,D,rd", [(8, 16, 128, 128), (3, 32, 64, 48), (1, 64, 128, 64)])
def test_rope_append_prompt_parts_among_decode_rows(kvq, half, H, P, D, rd):
    rng = np.random.default_rng([H, P, D, rd, 7])
    check_rope_append(kvq, mixed(rng, H, P, D), rng, 5 * H, rd, half)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("H,P,D,rd", [(8, 16, 128, 128), (3, 64, 64, 32), (4, 32, 128, 96),
                                      (2, 64, 128, 128), (1, 16, 128, 64)])
def test_rope_append_prompts(kvq, half, H, P, D, rd):
    rng = np.random.default_rng([H, P, D, rd])
    check_rope_append(kvq, prompts(rng, H, P, D), rng, 2 * H + 1 if H == 3 else 2 * H, rd, half)


def test_append_prompts_bad_pages_and_requests(kvq):
    """Bad entries in a prompt's table and a bad request among prompts: the others'
    pages are written all the same."""
    H, P, D = 8, 16, 64
    rng = np.random.default_rng(21)
    s = prompts(rng, H, P, D)
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    table, lens = s.table.copy(), s.lens.copy()
    table[0, 5], table[4, 100] = s.NP, -3
    lens[2] = 1
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kx, vx], s.tok_start, lens, table)
    c, err = run_append(kvq, s, (kt, vt), lens=lens, table=table)
    assert err == kvq.ERRBIT_SEQLEN | kvq.ERRBIT_PAGE
    assert_cache(c, pools, scales)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("H,G,P,D,rd", [(2, 4, 16, 128, 128), (8, 4, 16, 128, 64), (3, 1, 64, 128, 96),
                                        (1, 8, 32, 64, 64), (5, 2, 64, 64, 16)])
def test_rope_append(kvq, half, H, G, P, D, rd):
    """K rotated and rounded once, q beside it; V bit for bit."""
    rng = np.random.default_rng([H, G, P, rd])
    n, before = [1, 40, 0, 3, 1], [0, 10, 5, 30, 2000]
    check_rope_append(kvq, R.Step(rng, n, np.add(n, before), H, P, D, pad=2), rng, G * H, rd, half)


def check_rope_append(kvq, s, rng, Hq, rd, half):
    H, D = s.H, s.D
    (kt, kx), (vt, vx) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    q, qx = R.values(rng, s.N, Hq, D)
    f, m = inv_freq(rd, 500000.0), 1.1
    rope = kvq.Rope(dev(f), kvq.ROPE_HALF if half else kvq.ROPE_INTERLEAVED, m)
    c = cache_of(kvq, s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.full_like(q, 7.0).cuda()
    kvq.kvq_rope_block_append(c, rope, q.cuda(), qo, kt.cuda(), vt.cuda(), dev(s.tok_start),
                              dev(s.lens), dev(s.table), err_word=err)
    assert int(err.item()) == 0
    rows = int(s.tok_start[-1])
    pos = np.concatenate([np.arange(L - k, L) for k, L in zip(s.n, s.lens)])
    check_rotation(qo[:rows], qx[:rows], pos, f, half, m)
    assert (qo[rows:] == 7.0).all()
    kr = np.concatenate([R.rotate(kx[:rows], pos, f, half, m), kx[rows:]])
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    R.append(pools, scales, [kr, vx], s.tok_start, s.lens, s.table)
    got_k, got_s = c.k_pool.cpu().numpy(), c.scales.cpu().numpy()
    assert np.array_equal(c.v_pool.cpu().numpy(), pools[1])
    assert np.array_equal(got_s, scales)  # no amax of these inputs lies at a border
    # codes differ only where the rotation's error moves a value over a rounding
    # border, and then by one step of e4m3 (2^-3 of the value, 2^-9 scales below
    # 2^-6 scales)
    step = scales[:, :, 0][:, :, None, None].astype(np.float64)
    diff = got_k != pools[0]
    a, b = R.decode(got_k) * step, R.decode(pools[0]) * step
    assert diff.mean() < 1e-4
    assert (np.abs(a - b)[diff] <= (2.0 ** -3 * np.abs(b) + 2.0 ** -9 * step)[diff]).all()
    # in place: the same q
    q2 = q.cuda()
    kvq.kvq_rope_block_append(c, rope, q2, q2, kt.cuda(), vt.cuda(), dev(s.tok_start), dev(s.lens),
                              dev(s.table), err_word=err)
    assert torch.equal(q2[:rows], qo[:rows]) and np.array_equal(c.k_pool.cpu().numpy(), got_k)


# ---------------------------------------------------------------------------
# reading back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("H,P,D", SHAPES)
def test_read_is_exact(kvq, H, P, D):
    rng = np.random.default_rng([H, P, D])
    n, first = np.array([5, 0, 70, 1, 33]), np.array([0, 3, 11, 64, 31])
    s = R.Step(rng, n, n + first, H, P, D, pad=4)
    both = torch.full((s.N, 2 * H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    c = cache_of(kvq, s)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_block_read(c, dev(s.tok_start), dev(first.astype(np.int32)), dev(s.table),
                       both[:, :H], both[:, H:], err_word=err)
    assert int(err.item()) == 0
    got = both.double().cpu().numpy()
    rows = int(s.tok_start[-1])
    assert (got[rows:] == 3.0).all()
    for b in range(s.B):
        r = slice(int(s.tok_start[b]), int(s.tok_start[b + 1]))
        at = np.arange(first[b], first[b] + n[b])
        for i, pool in enumerate((s.k, s.v)):
            want = R.gather(pool, s.scales, i, s.table[b], at) if n[b] else np.zeros((0, H, D))
            assert np.array_equal(got[r, i * H:(i + 1) * H], want), (b, i)


def test_read_errors_and_roundtrip(kvq):
    """Bad ranges and pages leave their rows; a value read back and appended
    again gives the same codes; first=None reads from position 0."""
    H, P, D = 2, 16, 128
    rng = np.random.default_rng(9)
    n = np.array([20, 8, 4, 30])
    s = R.Step(rng, n, n, H, P, D)
    table = s.table.copy()
    table[3, 0] = s.NP + 4
    first = np.array([0, s.MP * P - 7, -1, 0], dtype=np.int32)
    k = torch.full((s.N, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = cache_of(kvq, s)
    kvq.kvq_block_read(c, dev(s.tok_start), dev(first), dev(table), k, v, err_word=err)
    assert int(err.item()) == kvq.ERRBIT_POS | kvq.ERRBIT_PAGE
    g = k.double().cpu().numpy()
    assert (g[20:32] == 3.0).all() and (g[32:48] == 3.0).all()
    assert np.array_equal(g[:20], R.gather(s.k, s.scales, 0, s.table[0], np.arange(20)))
    assert np.array_equal(g[48:], R.gather(s.k, s.scales, 0, s.table[3], np.arange(16, 30)))
    # what an append stores comes back, and appended again gives the same cache
    (kt, _), (vt, _) = R.values(rng, s.N, H, D), R.values(rng, s.N, H, D)
    c, _ = run_append(kvq, s, (kt, vt))
    kvq.kvq_block_read(c, dev(s.tok_start), None, dev(s.table), k, v)
    # (a block whose scale has room to spare may take a smaller one)
    d, _ = run_append(kvq, s, (k.cpu(), v.cpu()))
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    kvq.kvq_block_read(d, dev(s.tok_start), None, dev(s.table), k2, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_steps_captured_in_a_graph_and_on_another_stream(kvq):
    """Rotate-and-append, replayed with new inputs in the same buffers, on a side
    stream."""
    H, P, D, B, Hq = 2, 16, 128, 4, 8
    rng = np.random.default_rng(10)
    s = R.Step(rng, [1] * B, [30] * B, H, P, D)
    c = cache_of(kvq, s)
    pools, scales = [s.k.copy(), s.v.copy()], s.scales.copy()
    f = inv_freq(D)
    rope = kvq.Rope(dev(f))
    k, v, q = (torch.zeros(B, h, D, dtype=torch.bfloat16, device="cuda") for h in (H, H, Hq))
    lens = dev(np.zeros(B, dtype=np.int32))
    table = dev(s.table)
    lens.fill_(1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        kvq.kvq_block_append(c, k, v, None, lens, table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_rope(rope, lens, q, q)
        kvq.kvq_block_append(c, k, v, None, lens, table)
    for t in range(1, 25):
        (kt, kx), (vt, vx) = R.values(rng, B, H, D), R.values(rng, B, H, D)
        k.copy_(kt.cuda())
        v.copy_(vt.cuda())
        lens.fill_(t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        R.append(pools, scales, [kx, vx], None, np.full(B, t, dtype=np.int32), s.table)
    assert_cache(c, pools, scales)
