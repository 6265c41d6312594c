"""kvq_pages_fork over a cluster of CTAs with forks that get nothing among those that are served, and sequences of
forks, acquisitions, releases and compactions, against pages_ref.py, every array equal."""
import numpy as np
import pytest
import torch

import pages_ref as S
from test_gpu_pages_shared import Both, i32

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


def grow(kvq, x, req, first, n):
    """Pages for several requests by kvq_pages_update; those behind the first that does not fit get none."""
    ok, err = torch.full((len(req),), 9, dtype=torch.uint8, device="cuda"), i32([0])
    kvq.kvq_pages_update(x.state, acq_req=i32(req), acq_first=i32(first), acq_npages=i32(n), acq_ok=ok, err_word=err)
    want = np.cumsum(n) <= x.h.free_count[0]
    for b, f, m, w in zip(req, first, n, want):
        if w:
            S.acquire(x.h, b, f, m)
    x.same("acquire")
    assert np.array_equal(ok.cpu().numpy(), want) and (int(err.item()) == 0) == bool(want.all())
    return want


@pytest.mark.parametrize("seed", range(6))
def test_sequences_with_acquisitions(kvq, seed):
    """A run as a serving program makes it: prompts get pages, are forked, grow by pages of their own, end, and
    the pool is moved together; on one CTA and on many.  Acquisitions know nothing of holders."""
    rng = np.random.default_rng([51, seed])
    B, MP = ((12, 20), (40, 9), (300, 40), (25, 400), (900, 12), (60, 64))[seed]
    h = S.State(rng, B * MP // 3, B, MP)
    x = Both(kvq, h)
    tokens = np.zeros(B, dtype=np.int64)
    did = dict.fromkeys(("grow", "fork", "release"), 0)
    for step in range(16):
        pages = -(-tokens // P)
        idle, live = np.flatnonzero(pages == 0), np.flatnonzero(pages > 0)
        what = ("grow", "fork", "grow", "release")[step % 4]
        if what == "grow":
            req = rng.permutation(B)[:max(1, B // 4)]
            n = np.minimum(rng.integers(0, 1 + max(1, MP // 6), len(req)), MP - pages[req])
            got = grow(kvq, x, req, pages[req], n)
            tokens[req] = np.where(got & (n > 0), (pages[req] + n) * P - rng.integers(0, P, len(req)), tokens[req])
        elif what == "fork" and len(live) and len(idle):
            dst = rng.permutation(idle)[:max(1, len(idle) // 2)]
            src = rng.choice(live, len(dst))
            tok = (tokens[src] * rng.random(len(dst))).astype(np.int64)
            tok[::2] = tokens[src[::2]]
            got = x.fork(src, dst, tok, P)[2]
            tokens[dst] = np.where(got, tok, 0)
        elif what == "release" and len(live):
            req = rng.permutation(live)[:max(1, len(live) // 2)]
            keep = np.where(rng.random(len(req)) < 0.5, 0, pages[req] // 2)
            assert x.release(req, keep, pages[req] - keep) == 0
            tokens[req] = np.minimum(tokens[req], keep * P)
        did[what] += 1
        if step % 5 == 4:
            x.compact(-(-tokens // P))
        assert np.array_equal(x.h.shares, np.maximum(S.holders(x.h) - 1, 0))
    assert all(did.values())
    left = np.flatnonzero(tokens)
    assert x.release(left, None, -(-tokens[left] // P)) == 0
    assert x.h.free_count[0] == x.h.num_pages and not x.h.shares.any()
