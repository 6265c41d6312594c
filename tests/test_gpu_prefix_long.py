"""kvq_block_prefix_attn over prefixes and own tokens of a million tokens and more, where what the tensor
cores' truncating additions lose in one sum would pass a bf16 rounding."""
import numpy as np
import pytest
import torch

import block_ref as R
import prefix_ref as X
from test_gpu_block_prefix import attend, compare

pytestmark = pytest.mark.gpu

P = 64


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32)).cuda()


def near_ties(rng, tokens, D):
    """(V codes [tokens, D], their mean rounded to bf16 [D]): every value positive, and the mean 2^-11 of itself
    above the middle between two bf16 values, so that it is rounded up, and down where a sum has lost more than that.
    The first 4,096 tokens are chosen so that each dim's sum is the one wanted."""
    v = torch.from_numpy(rng.integers(0, 0x7F, (tokens, D), dtype=np.uint8)).cuda()
    v[:4096] = 0
    total = np.zeros(D)
    for part in v.split(1 << 18):
        total += part.view(R.E4M3).double().sum(0).cpu().numpy()
    grid = R.decode(np.arange(0x7F, dtype=np.uint8))
    first = np.zeros((4096, D), dtype=np.uint8)
    ulp = 2.0 ** (np.floor(np.log2(total / tokens)) - 7)  # of a bf16 there
    tie = (np.ceil(total / tokens / ulp - 0.5) + 0.5) * ulp
    tie = np.where(tie < total / tokens, tie + ulp, tie)
    for d in range(D):
        left, at = tie[d] * (1 + 2.0 ** -11) * tokens - total[d], 0
        for code in range(0x7E, 0, -1):
            n = int(left // grid[code])
            first[at:at + n, d] = code
            left -= n * grid[code]
            at += n
        assert at <= 4096 and 0 <= left < 2.0 ** -8
        total[d] = tie[d] * (1 + 2.0 ** -11) * tokens - left  # multiples of 2^-9 below 2^53: exact to 2^-26 of 1
    v[:4096] = torch.from_numpy(first).cuda()
    mean = total / tokens
    assert (mean > tie * (1 + 2.0 ** -11.5)).all() and (mean < tie + ulp / 2).all()
    return v, torch.from_numpy(tie + ulp / 2)


@pytest.mark.parametrize("D,tokens,B,own,G", [
    (128, 1 << 20, 160, False, 4),  # rows of work enough that one CTA sums whole prefixes
    (64, 1 << 20, 160, False, 16),
    (64, 1 << 21, 76, False, 2),    # and fewer: a prefix is cut among CTAs
    (128, 1 << 20, 160, True, 1),   # own tokens, written without a merge
    (64, 1 << 21, 100, True, 1),
    (64, (1 << 20) - 300, 160, True, 2)])
def test_long_sums_are_rounded_between(kvq, D, tokens, B, own, G):
    """Queries are zeros, so that every weight is 1 and the output the mean of V, whatever the split.  Weights and
    V scales are powers of two, products and the sum of weights (below 2^24) exact, so that only the sums of values
    lose anything: 2^-27 a token over at most 32,768 tokens (2^-12), and at most 200 additions of such sums, 2^-24 each,
    and three products of the result; less than 2^-11.9, and the mean stands 2^-11 above the place where the
    rounding changes.  So the output is the mean's rounding, bit for bit."""
    rng = np.random.default_rng([D, tokens, B, own])
    v, want = near_ties(rng, tokens, D)
    pages = -(-tokens // P)
    pool = torch.zeros(pages * P, D, dtype=torch.uint8, device="cuda")
    pool[:tokens] = v
    pool[tokens:] = 0x7E  # behind the length
    cache = kvq.BlockKVCache(torch.zeros(pages, 1, P, D, dtype=torch.uint8, device="cuda"), pool.view(pages, 1, P, D),
                             torch.ones(pages, 1, 2, device="cuda"))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)
    q = torch.zeros(B, G, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full((B, G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    err = i32([0])
    groups = (None, None) if own else (i32(np.arange(B + 1)), i32([pages - 1] * B))
    ws = kvq.block_prefix_workspace(B, G, 1, D)
    ws.fill_(0xFF)
    kvq.kvq_block_prefix_attn(cache, q, i32(np.arange(B + 1)), i32([tokens] * B), table, *groups, out, ws,
                              max_q=17 if own else 1, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got = out.double().cpu()
    wrong = got != want
    assert not wrong.any(), (float(wrong.double().mean()), got[wrong][0], want.expand_as(got)[wrong][0])


def repeated(s, B):
    """The step's one request B times, each a group of its own: rows of work enough that a CTA has whole ones."""
    n = int(s.n[0])
    s.B, s.N = B, B * n
    s.n, s.lens, s.table = np.repeat(s.n, B), np.repeat(s.lens, B), np.repeat(s.table, B, 0)
    s.tok_start = np.arange(0, (B + 1) * n, n, dtype=np.int32)
    s.group_start, s.pre = np.arange(B + 1, dtype=np.int32), np.repeat(s.pre, B)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("own", [False, True])
def test_joined_sums(kvq, D, own):
    """Sums that are taken out in between and joined: maxima that rise and fall, V scales 2^60 apart from one
    stretch of the prefix to the next, NaN codes and pages outside the pool in the first or the last of them."""
    rng = np.random.default_rng([41, D, own])
    s = X.Step(rng, [(0, [(3, 90001)])] if own else [(90001 // P, [(3, 7)])], 1, P, D)
    at = np.arange(s.MP) * P
    for stretch, (k, v) in enumerate(((-2, 20), (1, -40), (0, 0), (2, 20))):
        pages = s.table[0, (at >= 25000 * stretch) & (at < 25000 * (stretch + 1))]
        pages = pages[pages >= 0]
        s.scales[pages, :, 0] *= np.float32(2.0 ** k)
        s.scales[pages, :, 1] *= np.float32(2.0 ** v)
    G, B = 2, 160
    q = R.values(rng, s.N, G, D)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5)
    n = s.N
    repeated(s, B)
    want, tol, qs = np.tile(want, (B, 1, 1)), np.tile(tol, (B, 1, 1)), q[0].repeat(B, 1, 1)
    kw = dict(max_q=9)
    if own:
        kw["groups"] = (None, None)
    out, err = attend(kvq, s, qs, **kw)
    assert err == 0
    compare(out, want, tol)
    for token in (100, 40000, 89000):
        page, slot = s.table[0, token // P], token % P
        was = s.v[page, 0, slot, 3]
        s.v[page, 0, slot, 3] = 0x7F
        out, err = attend(kvq, s, qs, **kw)
        s.v[page, 0, slot, 3] = was
        assert err == 0 and bool(out[:, :, 3].isnan().all())
        out[:, :, 3] = 0
        other = want.copy()
        other[:, :, 3] = 0
        compare(out, other, tol)
        table = s.table.copy()
        table[::2, token // P] = s.NP
        out, err = attend(kvq, s, qs, table=table, **kw)
        assert err == kvq.ERRBIT_PAGE
        other, none = want.reshape(B, n, G, D).copy(), tol.reshape(B, n, G, D).copy()
        other[::2], none[::2] = 0, 0
        compare(out, other.reshape(want.shape), none.reshape(tol.shape))
