"""Attention of a batch whose requests share prefixes, in 64 bits on the host, with the bound
of the kernel's error in each value; and the steps that its tests use."""
import numpy as np

import block_ref as R


def attend(pools, scales, q, tok_start, seq_lens, table, sm_scale, skip=()):
    """(out float64 [N, Hq, D] with NaN in rows of nobody, bound).  The tables of a group's
    requests name the same pages in front, so that each request is computed by itself.

    The bound: with A = sum_d |q_d k_d| the largest over the row's tokens, a score's products
    and sums (fp32, any order, with truncation) are off by at most 2^-18 A sm; q's two pieces
    (e4m3 and e5m2, on a scale where a row's largest value lies in [224, 448)) by 2^-21.8 of
    that value where a value is below 2^-13.8 of it, and else are exact.  A weight's relative
    error is that, twice (its own and the maximum's), 2^-20 for exponentials and scales, and in
    the values' sum 2^-11 for its rounding to f16, or 2^-25 where f16 is subnormal: the operand
    is w_j s_j 2^(7 - n) (s_j the V scale, at most rounded up to a power of two) with 2^n at
    most twice the row's largest w_j s_j, so that it loses at most 2^-31 max_i(w_i s_i) times
    the code's magnitude.  Sums of L terms: tensor cores add 16 at a time and truncate, (L / 16 + 64)
    2^-23, and fp32 sums of the denominator less.  Then the result is rounded to bf16: half a
    step, 2^-8 of it."""
    N, Hq, D = q.shape
    H = pools[0].shape[1]
    G = Hq // H
    B, MP = table.shape
    P = pools[0].shape[2]
    out = np.full((N, Hq, D), np.nan)
    tol = np.zeros((N, Hq, D))
    for b in range(B):
        r = R.rows_of(tok_start, seq_lens, b, MP * P, N)
        if b in skip or r is None:
            s0, s1 = (b, b + 1) if tok_start is None else (int(tok_start[b]), int(tok_start[b + 1]))
            if 0 <= s0 <= s1 <= N:
                out[s0:s1] = 0.0
            continue
        row, n, p0 = r
        L = p0 + n
        if n == 0:
            continue
        k, v = (R.gather(pools[i], scales, i, table[b], np.arange(L)) for i in range(2))
        sv = scales[table[b, np.arange(L) // P], :, 1].astype(np.float64)
        for i in range(n):
            see = p0 + i + 1
            for g in range(H):
                hs = slice(g * G, (g + 1) * G)
                qq = q[row + i, hs].astype(np.float64)  # [G, D]
                kk, vv, s = k[:see, g], v[:see, g], sv[:see, g]
                x = qq @ kk.T * sm_scale
                w = np.exp(x - x.max(1, keepdims=True))
                den = w.sum(1, keepdims=True)
                o = w @ vv / den
                ak, aq = np.abs(kk), np.abs(qq)
                top = aq.max(1, keepdims=True)
                score = np.max(aq @ ak.T, 1, keepdims=True) * 2.0 ** -18
                score += np.max((aq < 2.0 ** -13.8 * top) @ ak.T, 1, keepdims=True) * top * 2.0 ** -21.8
                score *= abs(sm_scale)
                lost = 2.0 ** -31 * (w * s).max(1, keepdims=True) / den * np.sum(np.abs(vv) / s[:, None], 0)
                rel = 2 * (2 * score + 2.0 ** -20) + 2.0 ** -11 + 2 * (L / 16 + 64) * 2.0 ** -23
                t = rel * (w @ np.abs(vv) / den) + lost
                out[row + i, hs] = o
                tol[row + i, hs] = t + 2.0 ** -8 * (np.abs(o) + t) + 1e-37
    return out, tol


class Step(R.Step):
    """A ragged step of groups: groups[g] = (pages of its prefix, [(rows, own tokens) ...]); a
    request's own tokens are what it holds behind the prefix, its rows among them."""

    def __init__(self, rng, groups, H, P, D, spare=3, extra_pages=0, pad=0):
        members = [(g, n, own) for g, (_, reqs) in enumerate(groups) for n, own in reqs]
        pre = np.array([p for p, _ in groups], dtype=np.int64)
        of = np.array([g for g, _, _ in members], dtype=np.int64)
        lens = [int(pre[g]) * P + own for g, _, own in members]
        super().__init__(rng, [n for _, n, _ in members], lens, H, P, D, spare, extra_pages, pad)
        self.of, self.pre = of, pre.astype(np.int32)
        self.group_start = np.concatenate([[0], np.cumsum([len(r) for _, r in groups])]).astype(np.int32)
        for b in range(self.B):  # the first request's pages; the ones drawn for the others are spare
            lead = self.group_start[of[b]]
            self.table[b, :pre[of[b]]] = self.table[lead, :pre[of[b]]]
