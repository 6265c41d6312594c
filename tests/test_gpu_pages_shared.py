"""Pages that several requests hold: forks, releases, compaction and page copies against
the one-after-another forms of pages_ref.py, every array equal."""
import numpy as np
import pytest
import torch

import block_ref as R
import pages_ref as S

pytestmark = pytest.mark.gpu


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()


def i32(x):
    return dev(np.asarray(x, dtype=np.int32))


class Both:
    """The state on the host and on the GPU."""

    def __init__(self, kvq, host):
        self.kvq, self.h = kvq, host
        self.upload()
        self.ws = kvq.pages_workspace(host.num_pages, len(host.block_table))
        self.ws.fill_(0xFF)  # its contents need no preparation

    def upload(self):
        self.d = {n: dev(getattr(self.h, n)) for n in S.State.NAMES}
        d = self.d
        self.state = self.kvq.PageState(d["free_stack"], d["free_count"], d["page_tags"],
                                        d["block_table"], d["expected_tags"])

    def same(self, what):
        torch.cuda.synchronize()
        for n in S.State.NAMES:
            want = getattr(self.h, n)
            got = self.d[n].cpu().numpy().view(want.dtype)
            assert np.array_equal(got, want), (what, n)

    def fork(self, src, dst, tokens, P):
        n = len(src)
        cs, cd = i32(np.full(n, 77)), i32(np.full(n, 77))
        ok, err = torch.full((n,), 9, dtype=torch.uint8, device="cuda"), i32([0])
        self.kvq.kvq_pages_fork(self.state, self.d["shares"], i32(src), i32(dst), i32(tokens), P, cs, cd,
                                ok, self.ws, err_word=err)
        want = S.fork(self.h, src, dst, tokens, P)
        self.same("fork")
        got = cs.cpu().numpy(), cd.cpu().numpy(), ok.cpu().numpy(), int(err.item())
        for g, w in zip(got, want):
            assert np.array_equal(g, w), (g, w)
        return want

    def release(self, req, first, npages):
        err = i32([0])
        self.kvq.kvq_pages_release(self.state, self.d["shares"], i32(req), None if first is None else i32(first),
                                   i32(npages), self.ws, err_word=err)
        want = S.release(self.h, list(req), None if first is None else list(first), list(npages))
        self.same("release")
        assert (int(err.item()) != 0) == (want != 0) and int(err.item()) & want == want, (err, want)
        return int(err.item())

    def compact(self, held, cap=None):
        cap = self.h.num_pages // 2 if cap is None else cap
        cs, cd, moves, err = i32(np.full(cap, 77)), i32(np.full(cap, 77)), i32([77]), i32([0])
        self.kvq.kvq_pages_compact(self.state, self.d["shares"], i32(held), cs, cd, moves, self.ws,
                                   err_word=err)
        want = S.compact(self.h, list(held), cap)
        self.same("compact")
        assert np.array_equal(cs.cpu().numpy(), want[0]) and np.array_equal(cd.cpu().numpy(), want[1])
        assert int(moves.item()) == want[2]
        assert int(err.item()) == want[3]
        return want


def started(kvq, rng, num_pages, B, MP, counts):
    h = S.State(rng, num_pages, B, MP)
    for b, n in enumerate(counts):
        S.acquire(h, b, 0, n)
    return Both(kvq, h)


@pytest.mark.parametrize("seed", range(6))
def test_random_sequences(kvq, seed):
    """Forks, releases of whole requests and of tails, and compactions in turn."""
    rng = np.random.default_rng(seed)
    P, B, MP = (16, 32, 64)[seed % 3], int(rng.integers(4, 40)), int(rng.integers(2, 30))
    num = int(rng.integers(B * MP // 3, B * MP))
    x = started(kvq, rng, max(num, 4 * MP), B, MP, [MP, MP // 2, 1])
    length = np.zeros(B, dtype=np.int64)  # tokens
    length[:3] = [MP * P, (MP // 2) * P, min(5, P)]
    served = 0
    for step in range(14):
        live, idle = np.flatnonzero(length > 0), np.flatnonzero(length == 0)
        if step % 3 != 2 and len(live) and len(idle):
            k = int(rng.integers(1, len(idle) + 1))
            dst = rng.permutation(idle)[:k]
            src = rng.choice(live, k)
            tok = np.array([int(rng.integers(0, length[a] + 1)) for a in src])
            _, _, ok, _ = x.fork(src, dst, tok, P)
            length[dst] = np.where(ok, tok, 0)
            served += int(ok.sum())
        elif len(live):
            k = int(rng.integers(1, len(live) + 1))
            req = rng.permutation(live)[:k]
            pages = -(-length[req] // P)
            keep = (pages * rng.integers(0, 2, k) * rng.random(k)).astype(np.int64)
            assert x.release(req, keep, pages - keep) == 0
            length[req] = np.minimum(length[req], keep * P)
        if step % 4 == 3:
            x.compact(-(-length // P))
        held = S.holders(x.h)
        assert np.array_equal(x.h.shares, np.maximum(held - 1, 0))
    assert served > 0


def test_many_forks_and_the_stack_runs_out(kvq):
    """More forks than a round of 1,024, over both cluster sizes; the last ones find nothing."""
    rng = np.random.default_rng(3)
    for B, MP, pages, spare in ((2600, 5, [5, 3, 4], 700), (1200, 1, [1], 5000)):
        x = started(kvq, rng, sum(pages) + spare, B, MP, pages)
        n = B - 3 - 40
        src = rng.integers(0, len(pages), n)
        tok = np.array([int(rng.integers(0, pages[a] * 16 + 1)) for a in src])
        tok[::7] = 16  # shared pages alone
        dst = 3 + rng.permutation(B - 3)[:n]
        cs, cd, ok, err = x.fork(src, dst, tok, 16)
        assert (err == 0) == (spare > n) and (0 < ok.sum() < n) == (spare < n)
        done = dst[ok == 1]
        assert x.release(done, None, -(-tok[ok == 1] // 16)) == 0
        x.compact(np.r_[pages, np.zeros(B - len(pages), dtype=int)])


def test_large_lists(kvq):
    """Items of several batches a thread, chunks that begin inside a request."""
    rng = np.random.default_rng(4)
    B, MP = 70, 1500
    x = started(kvq, rng, 6000, B, MP, [1500, 700, 1333])
    n = 60
    src = rng.integers(0, 3, n)
    held = np.array([1500, 700, 1333])
    tok = (held[src] * 16 * rng.random(n)).astype(int)
    dst = 5 + rng.permutation(B - 5)[:n]
    x.fork(src, dst, tok, 16)
    count = np.zeros(B, dtype=int)
    count[:3], count[dst] = held, -(-tok // 16)
    x.compact(count)
    req = np.r_[0, dst[:50], 2]
    first = np.r_[1, np.zeros(50, dtype=int), 700]
    assert x.release(req, first, count[req] - first) == 0
    count[req] = first
    x.compact(count, cap=6000)
    left = np.flatnonzero(count)
    assert x.release(left, None, count[left]) == 0
    assert x.h.free_count[0] == 6000 and not x.h.shares.any()
    assert sorted(x.h.free_stack) == list(range(6000))


def test_forks_that_get_nothing(kvq):
    """Bad requests, the same request twice, tokens past the table, entries that are no pages: the
    others of the call are served."""
    rng = np.random.default_rng(5)
    x = started(kvq, rng, 64, 10, 4, [4, 2])
    for src, dst, tok, bits in [
            ([0, 0, -1, 10, 0], [2, 3, 4, 5, 10], [64, 5, 5, 5, 5], S.REQ),
            ([0, 0, 0], [4, 4, 0], [16, 17, 3], S.REQ),  # dst twice; a request forked onto itself
            ([0, 5], [5, 6], [16, 16], S.REQ),  # a source that the call writes
            ([0, 0, 1], [5, 6, 7], [-1, 65, 20], S.POS),
            ([1, 0], [8, 9], [33, 50], S.PAGE)]:  # request 1 holds two pages
        assert x.fork(src, dst, tok, 16)[3] == bits


def test_stack_with_bad_entries_and_counts(kvq):
    rng = np.random.default_rng(6)
    for bad in (-5, 40, 1 << 30):
        x = started(kvq, rng, 40, 6, 4, [4])
        x.h.free_stack[x.h.free_count[0] - 2] = bad
        x.upload()
        _, cd, ok, err = x.fork([0, 0, 0], [1, 2, 3], [5, 20, 40], 16)
        assert err == S.PAGE and ok.all() and (cd == -1).sum() == 1
        x.compact([4, 0, 0, 0, 0, 0])
    for count in (-1, 41):
        x = started(kvq, rng, 40, 6, 4, [4])
        x.h.free_count[0] = count
        x.upload()
        assert x.fork([0, 0], [1, 2], [5, 20], 16)[3] == S.PAGE
        assert x.release([0], None, [4]) == S.PAGE
        assert x.compact([4, 0, 0, 0, 0, 0])[3] == S.PAGE


def test_releases_that_are_refused(kvq):
    """All or nothing, for every reason, with good entries in the same list."""
    rng = np.random.default_rng(7)
    x = started(kvq, rng, 64, 8, 6, [5, 3, 4])
    x.fork([0, 0], [4, 5], [48, 70], 16)
    for req, first, n, bits in [([0, 8], None, [1, 1], S.REQ), ([0, 4, 0], None, [1, 1, 1], S.REQ), ([-1], None, [1], S.REQ),
                                ([0, 1], [0, 4], [1, 3], S.POS), ([0, 1], [-1, 0], [2, 1], S.POS),
                                ([0, 1], None, [2, -1], S.POS), ([0, 1], None, [5, 4], S.PAGE),
                                ([0, 1], [2 ** 31 - 1, 0], [2 ** 31 - 1, 0], S.POS)]:
        assert x.release(req, first, n) & bits
    x.h.block_table[3, 0] = x.h.block_table[1, 0]  # an entry that the holders do not count
    x.upload()
    assert x.release([1, 3], None, [1, 1]) == S.PAGE
    x.h.block_table[3, 0] = 64
    x.upload()
    assert x.release([3], None, [1]) == S.PAGE
    x.h.free_count[0] = 63
    x.upload()
    assert x.release([1, 2], None, [3, 4]) == S.PAGE  # the stack has no room
    x.h.free_count[0] = 3
    x.upload()
    assert x.release([2, 1], [1, 0], [3, 0]) == 0  # and a range of nothing


def test_compactions_that_are_refused(kvq):
    rng = np.random.default_rng(8)
    x = started(kvq, rng, 64, 4, 6, [5, 3])
    assert x.compact([5, 3, 0, 7])[3] == S.POS
    assert x.compact([5, 3, 0, -1])[3] == S.POS
    assert x.compact([5, 4, 0, 0])[3] == S.PAGE  # -1 is no page
    x.h.free_stack[3] = x.h.free_stack[4]
    x.upload()
    assert x.compact([5, 3, 0, 0])[3] == S.PAGE  # free twice
    x = started(kvq, rng, 64, 4, 6, [5, 3])
    x.h.block_table[2, 0] = x.h.free_stack[0]
    x.upload()
    assert x.compact([5, 3, 1, 0])[3] == S.PAGE  # held and free


@pytest.mark.parametrize("num,B", [(1, 1), (2, 1), (31, 2), (32, 2), (33, 2), (4097, 9), (70000, 5)])
def test_compaction_sizes(kvq, num, B):
    """Pools of every size against the bit words, empty, full, and part-filled; pages that no table
    holds are in use as well."""
    rng = np.random.default_rng(num)
    for part in (0.0, 1.0, 0.4):
        mine = int(num * part) // B
        h = S.State(rng, num, B, max(1, mine))
        for b in range(B):
            S.acquire(h, b, 0, mine)
        if part == 0.4:
            h.free_count[0] -= min(3, int(h.free_count[0]))  # held by nobody's table
        x = Both(kvq, h)
        x.compact([mine] * B)
        assert x.compact([mine] * B)[2] == 0  # the second time nothing is left to move


@pytest.mark.parametrize("dtype,H,P,D", [("e4m3", 8, 16, 128), ("bf16", 3, 32, 64), ("e4m3", 1, 16, 64), ("block", 8, 16, 128),
                                         ("block", 3, 64, 64), ("block", 1, 16, 64), ("block", 5, 32, 128)])
def test_page_copies(kvq, dtype, H, P, D):
    rng = np.random.default_rng(9)
    for NP, n in ((40, 11), (3000, 1400), (9, 0)):
        shape = (NP, H, P, D) if dtype != "bf16" else (NP, H, P, 2 * D)
        k, v = (rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2))
        sc = rng.random((NP, H, 2)).astype(np.float32)
        ids = rng.permutation(NP)
        src, dst = ids[:n].astype(np.int32), ids[n:2 * n].astype(np.int32)
        if n > 4:
            src[3] = src[0]  # one page to two places
            src[1], dst[2] = -1, -7
            src[4] = dst[4]
        dk, dv = dev(k), dev(v)
        err = i32([0])
        if dtype == "block":
            ds = dev(sc)
            kvq.kvq_block_copy_pages(kvq.BlockKVCache(dk, dv, ds), i32(src), i32(dst), err_word=err)
        else:
            as_pool = (lambda t: t.view(torch.bfloat16)) if dtype == "bf16" else (lambda t: t)
            kvq.kvq_copy_pages(kvq.KVCache(as_pool(dk), as_pool(dv)), i32(src), i32(dst), err_word=err)
        torch.cuda.synchronize()
        good = (src >= 0) & (dst >= 0)
        for a in (k, v, sc):
            a[dst[good]] = a[src[good]]
        assert int(err.item()) == 0
        assert np.array_equal(dk.cpu().numpy(), k) and np.array_equal(dv.cpu().numpy(), v)
        if dtype == "block":
            assert np.array_equal(ds.cpu().numpy(), sc)


def test_page_copies_leave_bad_pages_out(kvq):
    rng = np.random.default_rng(10)
    k = rng.integers(0, 256, (6, 2, 16, 64), dtype=np.uint8)
    sc = np.ones((6, 2, 2), dtype=np.float32)
    for src, dst in (([6, 1], [2, 3]), ([0, 1], [1 << 30, 3])):
        for block in (True, False):
            dk, dv, err = dev(k), dev(k), i32([0])
            if block:
                kvq.kvq_block_copy_pages(kvq.BlockKVCache(dk, dv, dev(sc)), i32(src), i32(dst), err_word=err)
            else:
                kvq.kvq_copy_pages(kvq.KVCache(dk, dv), i32(src), i32(dst), err_word=err)
            torch.cuda.synchronize()
            want = k.copy()
            want[3] = k[1]
            assert int(err.item()) == S.PAGE
            assert np.array_equal(dk.cpu().numpy(), want) and np.array_equal(dv.cpu().numpy(), want)


def test_copies_past_four_gigabytes(kvq):
    """Byte offsets that pass 32 bits."""
    NP, H, P, D = 70000, 8, 64, 128
    k = torch.zeros((NP, H, P, D), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    sc = torch.ones((NP, H, 2), device="cuda")
    k[NP - 2], v[NP - 2], sc[NP - 2] = 5, 9, 3.0
    kvq.kvq_block_copy_pages(kvq.BlockKVCache(k, v, sc), i32([NP - 2, NP - 2]), i32([NP - 1, 1]))
    torch.cuda.synchronize()
    for p in (NP - 1, 1):
        assert bool((k[p] == 5).all()) and bool((v[p] == 9).all()) and bool((sc[p] == 3.0).all())
    assert not bool(k[NP - 3].any()) and not bool(k[2].any())


def test_on_a_stream_and_in_a_graph(kvq):
    """A captured fork, copy and release, replayed on new state, on a stream of its own."""
    rng = np.random.default_rng(11)
    h = S.State(rng, 300, 12, 8)
    for b, n in enumerate([8, 5]):
        S.acquire(h, b, 0, n)
    x = Both(kvq, h)
    saved = {n: t.clone() for n, t in x.d.items()}
    src, dst, tok = [0, 1, 0, 0], [4, 5, 6, 7], [100, 64, 128, 3]
    ds, dd, dt = i32(src), i32(dst), i32(tok)
    cs, cd, err = i32([0] * 4), i32([0] * 4), i32([0])
    ok = torch.zeros(4, dtype=torch.uint8, device="cuda")
    req, num = i32([5, 0, 7]), i32([4, 8, 1])
    cache = kvq.BlockKVCache(*(dev(rng.integers(0, 256, (300, 2, 16, 64), dtype=np.uint8)) for _ in range(2)),
                             dev(rng.random((300, 2, 2)).astype(np.float32)))
    first_k = cache.k_pool.clone()
    stream = torch.cuda.Stream()

    def steps():
        kvq.kvq_pages_fork(x.state, x.d["shares"], ds, dd, dt, 16, cs, cd, ok, x.ws, err_word=err)
        kvq.kvq_block_copy_pages(cache, cs, cd, err_word=err)
        kvq.kvq_pages_release(x.state, x.d["shares"], req, None, num, x.ws, err_word=err)

    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        steps()
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        steps()
    want_cs, want_cd, want_ok, _ = S.fork(x.h, src, dst, tok, 16)
    assert S.release(x.h, [5, 0, 7], None, [4, 8, 1]) == 0
    for _ in range(3):
        for n, t in saved.items():
            x.d[n].copy_(t)
        cache.k_pool.copy_(first_k)
        torch.cuda.synchronize()
        g.replay()
        x.same("replay")
        assert np.array_equal(cs.cpu().numpy(), want_cs) and np.array_equal(cd.cpu().numpy(), want_cd)
        assert np.array_equal(ok.cpu().numpy(), want_ok) and int(err.item()) == 0
        for a, b in zip(want_cs, want_cd):
            if a >= 0:
                assert torch.equal(cache.k_pool[int(b)], first_k[int(a)])


def test_binding_refuses_other_shapes(kvq):
    x = started(kvq, np.random.default_rng(12), 32, 4, 4, [2])
    d, two, one = x.d, i32([0, 1]), i32([0])
    ok = torch.zeros(2, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="dst"):
        kvq.kvq_pages_fork(x.state, d["shares"], two, one, two, 16, two, two, ok, x.ws)
    with pytest.raises(ValueError, match="shares"):
        kvq.kvq_pages_fork(x.state, d["shares"][:5], two, two, two, 16, two, two, ok, x.ws)
    with pytest.raises(ValueError, match="npages"):
        kvq.kvq_pages_release(x.state, d["shares"], two, None, one, x.ws)
    with pytest.raises(ValueError, match="held"):
        kvq.kvq_pages_compact(x.state, d["shares"], two, i32([0] * 16), i32([0] * 16), one, x.ws)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_pages_compact(x.state, d["shares"], i32([0] * 4), i32([0] * 15), i32([0] * 15), one, x.ws)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_pages_release(x.state, d["shares"], two, None, two, x.ws[:256])
    x.same("after refusals")


def test_decode_goes_on_after_fork_and_compaction(kvq):
    """A prompt appended, forked in the middle of a page, both continued by other tokens, the pool
    moved together: attention gives what separate requests give, and the tag check passes."""
    rng = np.random.default_rng(13)
    H, G, P, D, B, MP, NP = 2, 4, 16, 64, 4, 6, 24
    h = S.State(rng, NP, B, MP)
    S.acquire(h, 0, 0, 3)
    x = Both(kvq, h)
    cache = kvq.BlockKVCache(torch.zeros(NP, H, P, D, dtype=torch.uint8, device="cuda"),
                             torch.zeros(NP, H, P, D, dtype=torch.uint8, device="cuda"),
                             torch.ones(NP, H, 2, device="cuda"))
    k, _ = R.values(rng, 40, H, D)
    v, _ = R.values(rng, 40, H, D)
    starts = lambda b, n: i32([0] * (b + 1) + [n] * (B - b))  # noqa: E731

    def append(b, rows, length):
        lens = np.zeros(B, dtype=np.int32)
        lens[b] = length
        kvq.kvq_block_append(cache, k[rows].cuda(), v[rows].cuda(), starts(b, len(rows)), i32(lens), x.d["block_table"])

    append(0, list(range(37)), 37)
    cs, cd, ok, _ = x.fork([0, 0], [1, 2], [37, 20], P)
    kvq.kvq_block_copy_pages(cache, i32(cs), i32(cd))
    append(1, [38, 39], 39)
    append(2, [30], 21)
    append(0, [37], 38)
    held = [3, 3, 2, 0]
    mcs, mcd, moves, _ = x.compact(held)
    assert moves > 0
    kvq.kvq_block_copy_pages(cache, i32(mcs), i32(mcd))
    mask = torch.full((B,), 7, dtype=torch.uint8, device="cuda")
    lens = i32([38, 39, 21, 0])
    kvq.kvq_check_tags(x.d["block_table"], lens, P, x.d["page_tags"], x.d["expected_tags"], mask)
    assert mask.cpu().tolist() == [0, 0, 0, 0]
    q, _ = R.values(rng, B, H * G, D)
    out = torch.zeros(B, H * G, D, device="cuda")
    ws = kvq.block_workspace(B, 1, H * G, H, D)
    kvq.kvq_block_attn(cache, q.cuda(), None, lens, x.d["block_table"], out, ws)
    # the same three sequences, each in pages of its own
    alone = kvq.BlockKVCache(torch.zeros(9, H, P, D, dtype=torch.uint8, device="cuda"),
                             torch.zeros(9, H, P, D, dtype=torch.uint8, device="cuda"),
                             torch.ones(9, H, 2, device="cuda"))
    table = i32(np.arange(12).reshape(4, 3) % 9)
    for b, parts in enumerate(([range(37), [37]], [range(37), [38, 39]], [range(20), [30]])):
        at = 0
        for rows in parts:
            rows = list(rows)
            at += len(rows)
            lens1 = np.zeros(B, dtype=np.int32)
            lens1[b] = at
            kvq.kvq_block_append(alone, k[rows].cuda(), v[rows].cuda(), starts(b, len(rows)), i32(lens1), table)
    want = torch.zeros_like(out)
    kvq.kvq_block_attn(alone, q.cuda(), None, lens, table, want, ws)
    torch.cuda.synchronize()
    # request 2's last page was scaled for 37 tokens and holds 5 of them: its scale may be larger than
    # alone, by one rounding of a code (2^-4) at most in K or V
    assert torch.equal(out[[0, 1, 3]], want[[0, 1, 3]])
    assert float((out[2] - want[2]).norm() / want[2].norm()) < 0.1


def test_refusals_that_one_of_many_blocks_sees(kvq):
    """Long lists, of more requests than a round takes, with one mistake at either end or in the middle: all
    or nothing for the whole cluster, and it goes on afterwards."""
    rng = np.random.default_rng(14)
    B, MP = 1500, 24
    held = rng.integers(0, MP + 1, B)
    held[[0, 700, B - 1]] = 20
    x = started(kvq, rng, int(held.sum()) + 900, B, MP, held)
    order = rng.permutation(B)
    order = np.r_[0, order[(order != 0) & (order != 700) & (order != B - 1)], 700, B - 1]
    for b in (0, 700, B - 1):
        for j, entry, shares in ((19, -1, None), (0, x.h.num_pages, None), (7, None, -1)):
            page = x.h.block_table[b, j]
            if shares is not None:
                x.h.shares[page] = shares
            else:
                x.h.block_table[b, j] = entry
            x.upload()
            assert x.release(order, None, held[order]) == S.PAGE
            if shares is None:
                assert x.compact(held)[3] == S.PAGE
            x.h.shares[page], x.h.block_table[b, j] = 0, page
            x.upload()
        assert x.release(np.r_[order, b], None, np.r_[held[order], 1]) & S.REQ
        at = int(np.flatnonzero(order == b)[0])
        n = held[order]
        n[at] = MP + 1
        assert x.release(order, None, n) == S.POS
        assert x.compact(np.where(np.arange(B) == b, MP + 1, held))[3] == S.POS
    for at in (0, int(x.h.free_count[0]) - 1):
        was = x.h.free_stack[at]
        for bad in (x.h.num_pages, x.h.free_stack[at - 1] if at else x.h.free_stack[1]):
            x.h.free_stack[at] = bad
            x.upload()
            assert x.compact(held)[3] == S.PAGE
        x.h.free_stack[at] = was
        x.upload()
    assert x.release(order[1:1200], None, held[order[1:1200]]) == 0
    gone = np.zeros(B, dtype=bool)
    gone[order[1:1200]] = True
    held[gone] = 0
    x.compact(held)
    src = rng.choice(np.flatnonzero(held), 1100)
    x.fork(src, np.flatnonzero(gone)[:1100], (held[src] * 16 * rng.random(1100)).astype(int), 16)
