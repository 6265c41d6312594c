"""Plain implementations, in 64 bits on the host, of the block-scaled cache's
operators, written from their definitions, and the ragged steps that the
tests use.  Nothing here is shared with the library."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def decode(codes):
    """uint8 codes -> float64 values."""
    return torch.from_numpy(np.ascontiguousarray(codes)).view(E4M3).to(torch.float64).numpy()


def encode(x):
    """float64 -> the nearest e4m3 codes (ties to even), saturating; NaN -> 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    grid = decode(np.arange(0x7F, dtype=np.uint8))  # 0 .. 448, increasing
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(grid, a, side="left"), 1, 0x7E)
    lo = hi - 1
    up = (a - grid[lo] > grid[hi] - a) | ((a - grid[lo] == grid[hi] - a) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def block_scale(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while 448.0 * s < amax:
        s *= 2.0
    return s


def rotate(x, pos, inv_freq, half, mscale=1.0):
    """x float64 [N, H, D] with its first 2 len(inv_freq) dims rotated.  Angles
    in extended precision: position times frequency has up to 84 bits."""
    rd = 2 * len(inv_freq)
    t = np.asarray(pos, dtype=np.longdouble)[:, None] * np.asarray(inv_freq, dtype=np.longdouble)
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    t = (t - np.floor(t / two_pi) * two_pi).astype(np.float64)
    c, s = mscale * np.cos(t)[:, None, :], mscale * np.sin(t)[:, None, :]
    y = np.array(x, dtype=np.float64)
    a_at = np.arange(rd // 2) if half else np.arange(0, rd, 2)
    b_at = a_at + rd // 2 if half else a_at + 1
    a, b = y[..., a_at].copy(), y[..., b_at].copy()
    y[..., a_at] = a * c - b * s
    y[..., b_at] = b * c + a * s
    return y


def rows_of(tok_start, seq_lens, b, cap, n_tokens):
    """(first row, rows, first position) of request b, or None if it is left out."""
    s0, s1 = (b, b + 1) if tok_start is None else (int(tok_start[b]), int(tok_start[b + 1]))
    if s0 < 0 or s1 < s0 or s1 > n_tokens:
        return None
    n, length = s1 - s0, int(seq_lens[b])
    if n and (length < n or length > cap):
        return None
    return s0, n, length - n


def append(pools, scales, new, tok_start, seq_lens, table):
    """pools: [k, v] uint8 [NP, H, P, D] and scales [NP, H, 2], changed in place;
    new: [k, v] float64 [N, H, D] (finite, inf or NaN)."""
    NP, H, P, _ = pools[0].shape
    B, MP = table.shape
    for b in range(B):
        r = rows_of(tok_start, seq_lens, b, MP * P, new[0].shape[0])
        if r is None:
            continue
        row, n, p0 = r
        for lp in range(p0 // P, (p0 + n - 1) // P + 1) if n else ():
            page = int(table[b, lp])
            if not 0 <= page < NP:
                continue
            lo, hi = max(p0, lp * P), min(p0 + n, lp * P + P)
            old = lo - lp * P
            for i in range(2):
                x = new[i][row + lo - p0:row + hi - p0]  # [tokens, H, D]
                for h in range(H):
                    v = np.abs(x[:, h])
                    s = block_scale(float(np.max(np.where(np.isfinite(v), v, 0.0))))
                    if old:
                        was = float(scales[page, h, i])
                        s = max(s, was)
                        if s > was:
                            pools[i][page, h, :old] = encode(decode(pools[i][page, h, :old]) * was / s)
                    scales[page, h, i] = s
                    pools[i][page, h, old:hi - lp * P] = encode(x[:, h] / s)


def gather(pool, scales, i, table_row, positions):
    """float64 [len(positions), H, D] values of cached tokens."""
    P = pool.shape[2]
    positions = np.asarray(positions, dtype=np.int64)
    page = np.asarray(table_row)[positions // P].astype(np.int64)
    return decode(pool[page, :, positions % P]) * scales[page, :, i].astype(np.float64)[:, :, None]


def attend(pools, scales, q, tok_start, seq_lens, table, sm_scale, skip=(), max_q=1):
    """(out float64 [N, Hq, D] with NaN in rows of nobody, bound of the kernel's
    error in each value).  skip: requests whose rows are zeros.

    The bound: with A = sum_d |q_d k_d| the largest over the row's tokens, a
    score's fp32 products and sums (128 terms, any order, with truncation) are
    off by at most 2^-18 A sm; a weight's relative error is that, twice (its own
    and the maximum's), plus 2^-21 (exponential) and 2^-21 (two f16 of a
    weight); sums of L terms in fp32, 16 at a time, add (L / 16 + 64) 2^-24.  The
    same for the denominator.  Below f16's smallest step a weight is lost: the
    operand of p.v is w_j s_j 2^(7 - n) (s_j the V scale, rounded up to a power
    of two) with 2^n at most twice the row's largest w_j s_j, and f16 rounds by
    at most 2^-25 near zero, so a token adds at most 2^-25 2^-7 2 max_i(w_i s_i)
    = 2^-31 max_i(w_i s_i) times its code's magnitude.

    With head_dim 128 and more than 16 rows (max_q times heads a kv head), or more
    than 8 where the table holds 4,096 tokens, both operands are sums of e4m3
    pieces.  A weight's four pieces, 2^5 apart, leave at most 2^-19 of it; the f16
    that holds what the first two leave is off by at most 2^-11 of 2^-10 of it, 2^-21,
    the f16 of the weight's own remainder by 2^-22 and the exponential and the sums by
    2^-21 and 2^-20: together below 2^-18; and 2^-10 2^-15 where e4m3 is subnormal, on a
    scale where the operand is w_j s_j 2^(1 - n): 2^-25 2^-1 2 max_i(w_i s_i) = 2^-25
    max_i(w_i s_i) a token.  q's two pieces, e4m3 and e5m2 on a scale where a row's
    largest value lies in [224, 448), are exact for values of 2^-6 and more there (what
    four bits leave of eight is at most eight units of the last place, and e5m2
    has three bits) and else off by 2^-14: values below 2^-13.8 of the largest are off by
    2^-21.8 of it.  The tensor core's sums are off by at most 2^-20 of the terms'
    magnitudes for 128 terms (scores: within the 2^-18 above; values: 2^-20 for each
    128 tokens' sum, on top of fp32's)."""
    N, Hq, D = q.shape
    H = pools[0].shape[1]
    G = Hq // H
    B, MP = table.shape
    P = pools[0].shape[2]
    out = np.full((N, Hq, D), np.nan)
    tol = np.zeros((N, Hq, D))
    for b in range(B):
        r = rows_of(tok_start, seq_lens, b, MP * P, N)
        if b in skip or r is None:
            s0, s1 = (b, b + 1) if tok_start is None else (int(tok_start[b]), int(tok_start[b + 1]))
            if 0 <= s0 <= s1 <= N:
                out[s0:s1] = 0.0
            continue
        row, n, p0 = r
        L = p0 + n
        if n == 0:
            continue
        k, v = (gather(pools[i], scales, i, table[b], np.arange(L)) for i in range(2))
        for i in range(n):
            see = p0 + i + 1
            for h in range(Hq):
                g = h // G
                qq = q[row + i, h].astype(np.float64)
                x = k[:see, g] @ qq * sm_scale
                w = np.exp(x - x.max())
                den = w.sum()
                out[row + i, h] = w @ v[:see, g] / den
                ak = np.abs(k[:see, g])
                score = np.max(ak @ np.abs(qq)) * abs(sm_scale) * 2.0 ** -18
                weight, floor = 2.0 ** -20, 2.0 ** -31
                if D == 128 and (max_q * G > 16 or (max_q * G > 8 and MP * P >= 4096)):
                    top = np.abs(qq).max()
                    score += np.max(ak @ (np.abs(qq) < 2.0 ** -13.8 * top)) * abs(sm_scale) * top * 2.0 ** -21.8
                    weight, floor = 2.0 ** -18, 2.0 ** -25
                s = scales[table[b, np.arange(see) // P], g, 1].astype(np.float64)
                lost = floor * (w * s).max() / den * np.sum(np.abs(v[:see, g]) / s[:, None], 0)
                rel = 2 * (2 * score + weight + (L / 16 + 64) * 2.0 ** -24)
                tol[row + i, h] = rel * (w @ np.abs(v[:see, g]) / den) + lost + 1e-30
    return out, tol


class Step:
    """A ragged step over a paged cache: requests of n[b] rows whose lengths after
    the step are lens[b], with shuffled pages and `spare` unused ones."""

    def __init__(self, rng, n, lens, H, P, D, spare=3, extra_pages=0, pad=0):
        self.n, self.lens = np.asarray(n, dtype=np.int32), np.asarray(lens, dtype=np.int32)
        self.B, self.H, self.P, self.D = len(self.n), H, P, D
        used = -(-self.lens.astype(np.int64) // P)
        self.MP = max(1, int(used.max(initial=0)) + extra_pages)
        self.NP = int(used.sum()) + spare
        ids = rng.permutation(self.NP)
        self.table = np.full((self.B, self.MP), -1, dtype=np.int32)
        at = 0
        for b in range(self.B):
            self.table[b, :used[b]] = ids[at:at + used[b]]
            at += int(used[b])
        self.tok_start = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.N = int(self.tok_start[-1]) + pad
        shape = (self.NP, H, P, D)
        self.k = rng.integers(0, 256, shape, dtype=np.uint8)
        self.v = rng.integers(0, 256, shape, dtype=np.uint8)
        for x in (self.k, self.v):  # no NaN codes
            x[(x & 0x7F) == 0x7F] ^= 0x01
        self.scales = np.exp2(rng.integers(-9, -2, (self.NP, H, 2))).astype(np.float32)


def bf16(x):
    """float -> the nearest bf16, as a torch tensor."""
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def values(rng, *shape):
    """bf16 activations as (torch bf16, float64 of the same values)."""
    t = bf16(rng.standard_normal(shape) * np.exp2(rng.integers(-2, 3, shape[:-1] + (1,))))
    return t, t.to(torch.float64).numpy()
