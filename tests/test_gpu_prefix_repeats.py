"""kvq_block_prefix_attn under changing conditions: cold and warm caches, other work on the GPU, so that
the warps of a CTA run at other paces.  Every result has the same bits, and they are right."""
import numpy as np
import pytest
import torch

import block_ref as R
import prefix_ref as X
from test_gpu_block_prefix import attend, cache_of, compare, dev

pytestmark = pytest.mark.gpu

# (groups of (pages of the prefix, [(rows, own tokens), ...]), H, P, D, G, max_q): blocks of few rows, in which
# whole warps have none, of one row more than a warp's, and full ones; own tokens by either kernel
CASES = {
    "drafts": ([(3 + 29 * g, [(1 + (b + g) % 5, 8 + 83 * ((3 * b + g) % 8)) for b in range(8)]) for g in range(5)], 3, 32, 64, 6, 5),
    "three_rows": ([(900, [(1, 16), (1, 16), (1, 16)])], 8, 16, 64, 8, 1),
    "rows_of_a_warp_and_one": ([(9, [(6, 1 + 37 * (b % 6) + 5) for b in range(18)]) for _ in range(6)], 8, 64, 128, 6, 6),
    "own_tokens_of_few_rows": ([(0, [(1, 700), (3, 1500), (2, 90), (4, 4000)])], 2, 16, 128, 8, 33),
    "prompts": ([(37, [(300, 300), (129, 700), (1, 40)]), (5, [(33, 33), (260, 261)])], 2, 32, 128, 3, 300),
    "prompts_of_a_small_model": ([(50, [(200, 230), (31, 900), (65, 65)])], 3, 16, 64, 6, 200),
    "full_blocks": ([(300, [(1, 30)] * 64)], 2, 16, 128, 4, 17),
}


@pytest.mark.parametrize("name", CASES)
def test_same_bits_whatever_runs_beside(kvq, name):
    groups, H, P, D, G, max_q = CASES[name]
    rng = np.random.default_rng([40, D, H])
    s = X.Step(rng, groups, H, P, D)
    q = R.values(rng, s.N, H * G, D)
    want, tol = X.attend([s.k, s.v], s.scales, q[1], s.tok_start, s.lens, s.table, D ** -0.5)
    cache, qd = cache_of(kvq, s), q[0].cuda()
    ws = kvq.block_prefix_workspace(s.N, H * G, H, D)
    args = [dev(x) for x in (s.tok_start, s.lens, s.table, s.group_start, s.pre)]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")  # twice the L2
    x = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    beside = torch.cuda.Stream()
    first, err = attend(kvq, s, qd, max_q=max_q, cache=cache)
    assert err == 0
    compare(first, want, tol)
    outs = [first.clone() for _ in range(150)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        if i % 3 == 1:
            flush.fill_(i)
        if i % 3 == 2:
            with torch.cuda.stream(beside):
                x @ x
        kvq.kvq_block_prefix_attn(cache, qd, *args, out, ws, max_q=max_q)
        if i % 2:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    other = [i for i, o in enumerate(outs) if not torch.equal(o.view(torch.int16), first.view(torch.int16))]
    assert not other, other
