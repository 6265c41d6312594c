"""Plain implementations of the calls for pages that several requests hold, one
request and one page after another, written from their definitions; nothing here is
shared with the library."""
import numpy as np

PAGE, POS, REQ, EXHAUSTED = 1, 4, 8, 32


class State:
    """The allocator's arrays on the host."""

    NAMES = ("free_stack", "free_count", "page_tags", "shares", "block_table", "expected_tags")

    def __init__(self, rng, num_pages, B, MP):
        self.free_stack = rng.permutation(num_pages).astype(np.int32)
        self.free_count = np.array([num_pages], dtype=np.int32)
        self.page_tags = rng.integers(0, 2 ** 32, num_pages, dtype=np.uint32)
        self.page_tags[::5] = 0xFFFFFFFF  # the next tag wraps
        self.shares = np.zeros(num_pages, dtype=np.int32)
        self.block_table = np.full((B, MP), -1, dtype=np.int32)
        self.expected_tags = np.zeros((B, MP), dtype=np.uint32)

    def copy(self):
        s = object.__new__(State)
        for n in self.NAMES:
            setattr(s, n, getattr(self, n).copy())
        return s

    @property
    def num_pages(self):
        return len(self.free_stack)

    def is_page(self, p):
        return 0 <= p < self.num_pages

    def bad_count(self):
        return not 0 <= self.free_count[0] <= self.num_pages


def acquire(s, b, first, n):
    """A request's pages, as kvq_pages_update hands them out."""
    for j in range(first, first + n):
        s.free_count[0] -= 1
        p = s.free_stack[s.free_count[0]]
        s.page_tags[p] += np.uint32(1)
        s.block_table[b, j], s.expected_tags[b, j] = p, s.page_tags[p]


def fork(s, src, dst, tokens, P):
    """(copy_src, copy_dst, ok, error bits); s changes in place."""
    n = len(src)
    B, MP = s.block_table.shape
    cs, cd, ok, err = np.full(n, -1, np.int32), np.full(n, -1, np.int32), np.zeros(n, np.uint8), 0
    if s.bad_count():
        return cs, cd, ok, PAGE
    whole = [0 <= a < B and 0 <= b < B and a != b for a, b in zip(src, dst)]
    writes = {b for b, w in zip(dst, whole) if w}
    seen, valid = set(), []
    for a, b, t, w in zip(src, dst, tokens, whole):
        good = w and b not in seen and a not in writes
        if w:
            seen.add(b)
        if not good:
            err |= REQ
        elif not 0 <= t <= MP * P:
            err, good = err | POS, False
        elif not all(s.is_page(p) for p in s.block_table[a, :-(-t // P)]):
            err, good = err | PAGE, False
        valid.append(good)
    out_of_pages = False
    for i in range(n):
        if not valid[i]:
            continue
        a, b, full, cut = src[i], dst[i], tokens[i] // P, tokens[i] % P > 0
        if out_of_pages or (cut and s.free_count[0] == 0):
            out_of_pages = True
            err |= EXHAUSTED
            continue
        ok[i] = 1
        for j in range(full):
            s.block_table[b, j], s.expected_tags[b, j] = s.block_table[a, j], s.expected_tags[a, j]
            s.shares[s.block_table[a, j]] += 1
        if cut:
            s.free_count[0] -= 1
            p = s.free_stack[s.free_count[0]]
            if not s.is_page(p):
                err |= PAGE
                continue
            s.page_tags[p] += np.uint32(1)
            s.block_table[b, full], s.expected_tags[b, full] = p, s.page_tags[p]
            cs[i], cd[i] = s.block_table[a, full], p
    return cs, cd, ok, err


def release(s, req, first, npages):
    """Error bits; s changes in place, or not at all.  The kernels raise a bit for what they
    have looked at when they stop, so only whether there is an error is compared."""
    B, MP = s.block_table.shape
    first = [0] * len(req) if first is None else first
    if s.bad_count():
        return PAGE
    if any(not 0 <= b < B for b in req) or len(set(req)) < len(req):
        return REQ
    if any(f < 0 or n < 0 or f + n > MP for f, n in zip(first, npages)):
        return POS
    t = s.copy()
    for b, f, n in zip(req, first, npages):
        for j in range(f, f + n):
            p = t.block_table[b, j]
            if not t.is_page(p) or t.shares[p] < 0:
                return PAGE
            t.block_table[b, j] = -1
            if t.shares[p] > 0:
                t.shares[p] -= 1
                continue
            if t.free_count[0] == t.num_pages or p in set(t.free_stack[s.free_count[0]:t.free_count[0]]):
                return PAGE
            t.free_stack[t.free_count[0]] = p
            t.free_count[0] += 1
    for n in State.NAMES:
        getattr(s, n)[...] = getattr(t, n)
    return 0


def compact(s, held, cap):
    """(copy_src, copy_dst, moves, error bits)"""
    none = np.full(cap, -1, np.int32), np.full(cap, -1, np.int32), 0
    B, MP = s.block_table.shape
    n = s.num_pages
    if s.bad_count():
        return (*none, PAGE)
    if any(not 0 <= h <= MP for h in held):
        return (*none, POS)
    free = [int(p) for p in s.free_stack[:s.free_count[0]]]
    if len(set(free)) < len(free) or not all(s.is_page(p) for p in free):
        return (*none, PAGE)
    used = set(range(n)) - set(free)
    if any(int(p) not in used for b in range(B) for p in s.block_table[b, :held[b]]):
        return (*none, PAGE)
    live = len(used)
    movers, holes = sorted(p for p in used if p >= live), sorted(p for p in free if p < live)
    cs, cd, _ = none
    cs[:len(movers)], cd[:len(holes)] = movers, holes
    to = dict(zip(movers, holes))
    for a, b in to.items():
        s.page_tags[b] += np.uint32(1)
        s.shares[b], s.shares[a] = s.shares[a], 0
    for b in range(B):
        for j in range(held[b]):
            p = int(s.block_table[b, j])
            if p in to:
                s.block_table[b, j], s.expected_tags[b, j] = to[p], s.page_tags[to[p]]
    s.free_stack[:len(free)] = range(n - 1, live - 1, -1)
    return cs, cd, len(movers), 0


def holders(s):
    """Table entries of each page."""
    t = s.block_table[s.block_table >= 0]
    return np.bincount(t, minlength=s.num_pages)
