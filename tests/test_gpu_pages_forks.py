"""kvq_pages_fork over a cluster of CTAs with forks that get nothing among those that are served, against
pages_ref.py, every array equal."""
import numpy as np
import pytest

import pages_ref as S
from test_gpu_pages_shared import Both

pytestmark = pytest.mark.gpu

P = 16


@pytest.mark.parametrize("seed", range(12))
def test_forks_of_many_blocks_that_get_nothing(kvq, seed):
    """Entries that are no pages in several sources, at either end of short and long ones, so that several CTAs
    find bad forks in the same round and in others; requests outside the batch, named twice, or written and read;
    tokens past the table; rounds of 1,024 forks whose pages do not divide evenly."""
    rng = np.random.default_rng([50, seed])
    B, MP, parents = 2700 + 13 * seed, int(rng.integers(12, 60)), 64
    held = rng.integers(1, MP + 1, parents)
    held[:4] = [MP, 1, MP, MP - 1]
    h = S.State(rng, int(held.sum()) + (400 if seed % 3 == 0 else 3000), B, MP)
    for b, n in enumerate(held):
        S.acquire(h, b, 0, n)
    for b in (0, 1, 5, 9, 17, 33, 40, 63)[:2 + seed % 7]:
        j = (0, held[b] - 1, held[b] // 2)[(b + seed) % 3]
        h.block_table[b, j] = (-1, h.num_pages, 1 << 30, -2 ** 31, 2 ** 31 - 1)[int(rng.integers(0, 5))]
    x = Both(kvq, h)
    n = B - parents - 7
    src = rng.integers(0, parents, n)
    src[rng.random(n) < 0.2] = 0  # many of one bad request, next to one another and apart
    dst = parents + rng.permutation(B - parents)[:n]
    tok = (held[src] * P * rng.random(n)).astype(np.int64)
    tok[::5] = held[src[::5]] * P
    tok[3::41] += P  # (an entry that the source does not hold, or past the table)
    if seed % 2:
        for k, (a, b, t) in enumerate([(-1, dst[0], 5), (B, dst[1], 5), (3, B, 5), (4, 4, 5), (2, dst[n // 2], 9),
                                       (dst[7], dst[8], 16), (3, dst[9], -1), (3, dst[10], MP * P + 1)]):
            at = (k * 331 + seed) % n
            src[at], dst[at], tok[at] = a, b, t
    cs, cd, ok, err = x.fork(src, dst, tok, P)
    assert err & S.PAGE and 0 < ok.sum() < n
    # and the state goes on: what was served is given back
    served = np.flatnonzero(ok)
    assert x.release(dst[served], None, -(-tok[served] // P)) == 0
