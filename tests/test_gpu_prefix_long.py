"""kvq_block_prefix_attn over prefixes and own tokens of a million tokens and more, where what the tensor
cores' truncating additions lose in one sum would pass a bf16 rounding."""
import numpy as np
import pytest
import torch

import block_ref as R

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
