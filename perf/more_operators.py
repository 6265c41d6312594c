"""Cases of pages that several requests share: forking a request, giving its pages
back, moving the pool's pages together, copying pages, and attention that reads a
prefix which a group of requests shares once for all of them.

Each case is one call that a serving program makes when it answers one prompt several
times, keeps a system prompt for many users, or searches over beams.  ``own`` false
computes it with elementary torch operations, true makes the framework's call.

The allocator's state is the framework's (a stack of free pages, a tag for each page that
changes when the page is handed out, block tables with the tags that their requests
expect), and one number more for each page: how many table entries hold it beyond the
first.  A pass of an allocator case starts from the same saved state, which it copies back
in both forms.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
UP = 64  # parts of a state begin at a multiple of so many numbers


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one prompt answered four times, from the middle of a page on: latency counts
        {"name": "fork_4_of_1", "op": "fork", "parents": 1, "forks": 4, "lo": 700, "hi": 700,
         "whole": True, "spare": 64, "p": 16, "mix": 1},
        # every request of a large batch forked, from prompts up to 32k
        {"name": "fork_256_of_16", "op": "fork", "parents": 16, "forks": 256, "lo": 500,
         "hi": 32768, "whole": False, "spare": 4096, "p": 16, "mix": 2},
        # rejected answers of one prompt end
        {"name": "release_3_of_8", "op": "release", "parents": 2, "forks": 6, "lo": 300, "hi": 2500,
         "own_hi": 200, "gone": 3, "tails": False, "p": 16, "mix": 3},
        # a whole batch of long answers to shared prompts ends, or drops its last pages
        {"name": "release_200_of_272", "op": "release", "parents": 16, "forks": 256, "lo": 500,
         "hi": 16384, "own_hi": 4000, "gone": 200, "tails": True, "p": 16, "mix": 4},
        # a small pool moved together
        {"name": "compact_2k_pages", "op": "compact", "pages": 2048, "b": 32, "held": 0.4,
         "shared": 0.3, "mix": 5},
        # a large one, mostly used
        {"name": "compact_300k_pages", "op": "compact", "pages": 300000, "b": 256, "held": 0.8,
         "shared": 0.5, "mix": 6},
        # the last, part-filled pages of forked requests
        {"name": "copy_48_pages", "op": "copy", "pages": 4096, "pairs": 48, "hkv": 8, "d": 128,
         "p": 16, "mix": 7},
        # what a compaction moves
        {"name": "copy_20k_pages", "op": "copy", "pages": 50000, "pairs": 20011, "hkv": 8,
         "d": 128, "p": 16, "mix": 8},
        # a few answers to one short prompt
        {"name": "attn_4_share_1k", "op": "attn", "b": 4, "groups": 1, "n_lo": 1, "n_hi": 1,
         "pre_lo": 1040, "pre_hi": 1040, "own_lo": 1, "own_hi": 60, "hq": 32, "hkv": 8, "d": 128,
         "p": 16, "pad": 0, "aborted": 0, "mix": 9},
        # many users behind one system prompt, answers of all lengths
        {"name": "attn_64_share_8k", "op": "attn", "b": 64, "groups": 1, "n_lo": 1, "n_hi": 1,
         "pre_lo": 8192, "pre_hi": 8192, "own_lo": 1, "own_hi": 1000, "hq": 32, "hkv": 8, "d": 128,
         "p": 16, "pad": 0, "aborted": 0, "mix": 10},
        # drafted tokens of a small model, several prompts, padded behind the last request
        {"name": "attn_drafts_d64_5_groups", "op": "attn", "b": 40, "groups": 5, "n_lo": 1,
         "n_hi": 5, "pre_lo": 96, "pre_hi": 6000, "own_lo": 8, "own_hi": 700, "hq": 18, "hkv": 3,
         "d": 64, "p": 32, "pad": 7, "aborted": 1, "mix": 11},
        # a large batch over one long document
        {"name": "attn_256_share_32k", "op": "attn", "b": 256, "groups": 1, "n_lo": 1, "n_hi": 1,
         "pre_lo": 32768, "pre_hi": 32768, "own_lo": 1, "own_hi": 700, "hq": 64, "hkv": 8,
         "d": 128, "p": 64, "pad": 0, "aborted": 0, "mix": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))))


def draw(rng):
    op = rng.choice(["fork", "release", "compact", "copy", "attn", "attn", "attn"])
    p = rng.choice([16, 32, 64])
    mix = rng.randrange(1 << 20)
    if op == "fork":
        hi = _log_int(rng, 1, 30000)
        return {"op": op, "parents": _log_int(rng, 1, 16), "forks": _log_int(rng, 1, 250),
                "lo": rng.choice([1, max(1, hi // 20), hi]), "hi": hi, "whole": rng.random() < 0.3,
                "spare": rng.choice([3, 500]), "p": p, "mix": mix}
    if op == "release":
        parents, forks = _log_int(rng, 1, 16), _log_int(rng, 1, 250)
        hi = _log_int(rng, 1, 16000)
        return {"op": op, "parents": parents, "forks": forks, "lo": rng.choice([1, hi]), "hi": hi,
                "own_hi": _log_int(rng, 1, 3900), "gone": rng.randint(1, parents + forks),
                "tails": rng.random() < 0.5, "p": p, "mix": mix}
    if op == "compact":
        return {"op": op, "pages": _log_int(rng, 9, 290000), "b": _log_int(rng, 1, 250),
                "held": round(rng.uniform(0.05, 0.95), 3), "shared": rng.choice([0.0, 0.3, 0.6]),
                "mix": mix}
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    if op == "copy":
        pages = _log_int(rng, 8, 400000 // hkv // p)
        return {"op": op, "pages": pages, "pairs": _log_int(rng, 1, pages // 2), "hkv": hkv, "d": d,
                "p": p, "mix": mix}
    b = _log_int(rng, 1, 160)
    groups = rng.randint(1, min(b, 6))
    n_hi = rng.choice([1, 1, rng.randint(2, 8)])
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 6, 8])
    hi = _log_int(rng, p, min(24000 // groups, 256 * 64 * 30000 // (b * n_hi * hq)))
    own_hi = _log_int(rng, n_hi, min(3000, 60000 // b))
    return {"op": op, "b": b, "groups": groups, "n_lo": rng.choice([1, n_hi]), "n_hi": n_hi,
            "pre_lo": rng.choice([0, hi // 8, hi]), "pre_hi": hi,
            "own_lo": rng.choice([1, own_hi]), "own_hi": own_hi,
            "hq": hq, "hkv": hkv, "d": d, "p": p, "pad": rng.choice([0, rng.randint(1, 9)]),
            "aborted": rng.choice([0, 0, 1]), "mix": mix}


def _spread(r, lo, hi, n):
    """n whole numbers of [lo, hi], spread over their logarithm; both ends among them."""
    a = np.exp(r.uniform(np.log(lo + 1), np.log(hi + 1), n)) - 1
    a = np.clip(np.round(a), lo, hi).astype(np.int64)
    if n > 1:
        a[0], a[n - 1] = hi, lo
    return a


def _fork_plan(case):
    """Lengths of the parents; source, slot and tokens of every fork."""
    r = np.random.RandomState(case["mix"])
    k, n = case["parents"], case["forks"]
    lens = _spread(r, case["lo"], case["hi"], k)
    src = r.randint(0, k, n)
    dst = k + r.permutation(n)
    tok = lens[src] if case["whole"] else np.maximum(1, (lens[src] * r.rand(n)).astype(np.int64))
    return lens, src, dst, tok


def _release_plan(case):
    """Parents' pages, forks' source, shared and own pages; who gives back what."""
    r = np.random.RandomState(case["mix"])
    k, n, p = case["parents"], case["forks"], case["p"]
    pages = -(-_spread(r, case["lo"], case["hi"], k) // p)
    src = r.randint(0, k, n)
    part = (pages[src] * r.rand(n)).astype(np.int64)
    mine = -(-_spread(r, 1, case["own_hi"], n) // p)
    held = np.concatenate([pages, part + mine])
    who = r.permutation(k + n)[:case["gone"]]
    first = (held[who] * r.rand(len(who)) * (r.rand(len(who)) < 0.5)).astype(np.int64)
    if not case["tails"]:
        first[:] = 0
    return pages, src, part, mine, who, first, held[who] - first


def _compact_plan(case):
    """Pages of every request: (shared with the first one, its own)."""
    r = np.random.RandomState(case["mix"])
    live = max(1, int(case["pages"] * case["held"]))
    cut = np.sort(r.randint(0, live + 1, case["b"] - 1))
    mine = np.diff(np.concatenate([[0], cut, [live]]))
    part = (mine[0] * r.rand(case["b"]) * (r.rand(case["b"]) < case["shared"])).astype(np.int64)
    part[0] = 0
    return part, mine


def _attn_plan(case):
    """Rows of every request, groups' first requests, their prefix pages, lengths."""
    r = np.random.RandomState(case["mix"])
    b, k, p = case["b"], case["groups"], case["p"]
    n = r.randint(case["n_lo"], case["n_hi"] + 1, b).astype(np.int64)
    at = np.concatenate([[0], np.sort(r.permutation(b - 1)[:k - 1]) + 1, [b]]).astype(np.int64)
    pre = _spread(r, case["pre_lo"], case["pre_hi"], k) // p
    of = np.repeat(np.arange(k), np.diff(at))
    mine = np.maximum(_spread(r, case["own_lo"], case["own_hi"], b), n)
    return n, at, pre, of, pre[of] * p + mine


def _aborted(case):
    """The request that the tag check aborted, if one was."""
    return case["b"] // 2 if case["aborted"] else -1


def work(case):
    op = case["op"]
    if op == "fork":
        _, src, _, tok = _fork_plan(case)
        full = tok // case["p"]
        distinct = sum(int(full[src == k].max()) for k in np.unique(src))
        # entry and tag read and written, the holders of every page; a fork's lists, a new page
        by = 16 * int(full.sum()) + 8 * distinct + len(src) * (12 + 9) + 24 * int((tok % case["p"] > 0).sum())
        return {"bytes": by, "flops": int(full.sum())}
    if op == "release":
        _, _, _, _, who, _, n = _release_plan(case)
        # an entry read and cleared, the holders of its page, and the page on the stack
        return {"bytes": int(n.sum()) * (8 + 8 + 4) + 12 * len(who), "flops": int(n.sum())}
    if op == "compact":
        part, mine = _compact_plan(case)
        n, live = case["pages"], int(mine.sum())
        moves = min(live, n - live) * max(live, n - live) // n  # of random pages, about so many
        # the free stack read and written, the tables read, what moves written
        by = 8 * (n - live) + 4 * int((part + mine).sum()) + moves * (8 + 8 + 8 + 8)
        return {"bytes": by, "flops": n}
    if op == "copy":
        page = 2 * case["hkv"] * (case["p"] * case["d"] + 4)
        return {"bytes": case["pairs"] * (2 * page + 8), "flops": 0}
    n, at, pre, of, total = _attn_plan(case)
    live = np.arange(case["b"]) != _aborted(case)
    h, d, p = case["hkv"], case["d"], case["p"]
    mine = (total - pre[of] * p) * live
    seen = (n * total - n * (n - 1) // 2) * live
    tokens = int(pre.sum()) * p + int(mine.sum())
    pages = int(pre.sum()) + int(np.sum(-(-mine // p)))
    return {"bytes": tokens * 2 * h * d + pages * (8 * h + 4) + int(n.sum()) * case["hq"] * d * 4,
            "flops": 4 * int(seen.sum()) * case["hq"] * d}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).to(DEV)


def _rand(g, n):
    return torch.randperm(n, generator=g, device=DEV).to(torch.int32)


def _state(pages, free, tags, shares, table):
    """The allocator's state in one buffer, saved and live."""
    b, mp = table.shape
    stack = torch.zeros(pages, dtype=torch.int32, device=DEV)
    stack[:free.numel()] = free
    count = torch.tensor([free.numel()], dtype=torch.int32, device=DEV)
    expected = torch.where(table >= 0, tags[table.clamp(min=0).long()], 0)
    parts = {"free_stack": stack, "free_count": count, "page_tags": tags, "shares": shares,
             "block_table": table, "expected_tags": expected}
    saved = torch.cat([torch.nn.functional.pad(x.flatten(), (0, -x.numel() % UP))
                       for x in parts.values()])
    live, at, s = saved.clone(), 0, {"saved": saved}
    for name, x in parts.items():
        s[name] = live[at:at + x.numel()].view(x.shape)
        at += x.numel() + -x.numel() % UP
    s["live"] = live
    return s


def _tags(g, pages):
    return torch.randint(-2 ** 31, 2 ** 31, (pages,), generator=g, device=DEV).to(torch.int32)


def _columns(mp):
    return torch.arange(mp, device=DEV)[None, :]


def _with_shared(perm, part, mine, leader, mp):
    """Tables of requests that hold the first `part` pages of their leader and then `mine` of
    their own, taken from `perm`; a leader holds pages of its own alone."""
    b = len(mine)
    own_ = torch.full((b, mp), -1, dtype=torch.int32, device=DEV)
    part_, mine_ = _dev(part)[:, None], _dev(mine)[:, None]
    col = _columns(mp)
    here = (col >= part_) & (col < part_ + mine_)
    own_[here] = perm[:int(mine.sum())]
    return torch.where(col < part_, own_[_dev(leader).long()], own_)


def _prepare_fork(case, g):
    lens, src, dst, tok = _fork_plan(case)
    pages = -(-lens // case["p"])
    b, mp = case["parents"] + case["forks"], int(pages.max())
    used = int(pages.sum())
    perm = _rand(g, used + case["spare"])
    zero = np.zeros(case["forks"], dtype=np.int64)
    mine = np.concatenate([pages, zero])
    table = _with_shared(perm, 0 * mine, mine, 0 * mine, mp)
    n = used + case["spare"]
    s = _state(n, perm[used:], _tags(g, n), torch.zeros(n, dtype=torch.int32, device=DEV), table)
    k = len(src)
    s |= {"src": _dev(src), "dst": _dev(dst), "tokens": _dev(tok),
          "copy_src": torch.zeros(k, dtype=torch.int32, device=DEV),
          "copy_dst": torch.zeros(k, dtype=torch.int32, device=DEV),
          "ok": torch.zeros(k, dtype=torch.uint8, device=DEV)}
    return s


def _holders(table, pages):
    """Table entries that hold each page."""
    at = torch.where(table >= 0, table, pages).long().flatten()
    count = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)
    return count.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:pages]


def _prepare_release(case, g):
    pages, src, part, mine, who, first, n = _release_plan(case)
    k = case["parents"]
    part = np.concatenate([0 * pages, part])
    mine = np.concatenate([pages, mine])
    used = int(mine.sum())
    total = used + used // 4 + 1
    perm = _rand(g, total)
    leader = np.concatenate([np.arange(k), src])
    table = _with_shared(perm, part, mine, leader, int((part + mine).max()))
    shares = (_holders(table, total) - 1).clamp(min=0).to(torch.int32)
    s = _state(total, perm[used:], _tags(g, total), shares, table)
    return s | {"req": _dev(who), "first": _dev(first), "npages": _dev(n)}


def _prepare_compact(case, g):
    part, mine = _compact_plan(case)
    total, used = case["pages"], int(mine.sum())
    perm = _rand(g, total)
    table = _with_shared(perm, part, mine, 0 * mine, max(1, int((part + mine).max())))
    shares = (_holders(table, total) - 1).clamp(min=0).to(torch.int32)
    s = _state(total, perm[used:], _tags(g, total), shares, table)
    return s | {"held": _dev(part + mine),
                "copy_src": torch.zeros(total, dtype=torch.int32, device=DEV),
                "copy_dst": torch.zeros(total, dtype=torch.int32, device=DEV),
                "moves": torch.zeros(1, dtype=torch.int32, device=DEV)}


def _pool(g, pages, h, p, d):
    """A pool as a run of the cache leaves it: codes and scales of random pages."""
    codes = torch.empty(pages, h, p, d, dtype=torch.uint8, device=DEV)
    exp = torch.empty(pages, h, device=DEV)
    step = max(1, (1 << 27) // (h * p * d))
    for at in range(0, pages, step):
        x = torch.randn(min(step, pages - at), h, p, d, generator=g, device=DEV)
        x *= torch.exp2(torch.randint(-3, 4, (x.shape[0], h, 1, 1), generator=g, device=DEV).float())
        e = torch.ceil(torch.log2(x.abs().amax((2, 3)) / E4M3_MAX))
        codes[at:at + step] = (x * torch.exp2(-e)[:, :, None, None]).clamp_(-448, 448) \
            .to(torch.float8_e4m3fn).view(torch.uint8)
        exp[at:at + step] = e
    return codes.view(torch.float8_e4m3fn), torch.exp2(exp)


def _values(g, shape):
    """bf16 activations: heads of different size, some large values."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-3, 4, (shape[-2], 1), generator=g, device=DEV).float())
    x *= torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.02, 12.0, 1.0)
    return x.to(torch.bfloat16)


def _prepare_copy(case, g):
    s = {}
    s["k_pool"], ks = _pool(g, case["pages"], case["hkv"], case["p"], case["d"])
    s["v_pool"], vs = _pool(g, case["pages"], case["hkv"], case["p"], case["d"])
    s["scales"] = torch.stack([ks, vs], dim=2).contiguous()
    perm = _rand(g, case["pages"])
    n = case["pairs"]
    return s | {"copy_src": perm[:n].contiguous(), "copy_dst": perm[n:2 * n].contiguous()}


def _prepare_attn(case, g):
    n, at, pre, of, total = _attn_plan(case)
    h, p, d, b = case["hkv"], case["p"], case["d"], case["b"]
    mine = -(-(total - pre[of] * p) // p)
    k = case["groups"]
    # a row of its own for each group's prefix, then the requests
    count = np.concatenate([pre, mine])
    part = np.concatenate([0 * pre, pre[of]])
    leader = np.concatenate([np.arange(k), of])
    pages = int(count.sum()) + int(count.sum()) // 20 + 1
    table = _with_shared(_rand(g, pages), part, count, leader, int((part + count).max()))
    start = np.concatenate([[0], np.cumsum(n)])
    s = {"block_table": table[k:].contiguous(), "tok_start": _dev(start), "seq_lens": _dev(total),
         "group_start": _dev(at), "prefix_pages": _dev(pre)}
    s["k_pool"], ks = _pool(g, pages, h, p, d)
    s["v_pool"], vs = _pool(g, pages, h, p, d)
    s["scales"] = torch.stack([ks, vs], dim=2).contiguous()
    rows = int(start[-1]) + case["pad"]
    s["q"] = _values(g, (rows, case["hq"], d))
    s["out"] = torch.zeros(rows, case["hq"], d, dtype=torch.bfloat16, device=DEV)
    s["n_max"] = int(n.max())
    # what the plain form pads to: rows of a group, pages of a prefix and of a request's own
    s["most"] = (int((start[at[1:]] - start[at[:-1]]).max()), max(1, int(pre.max())), int(mine.max()))
    s["abort"] = torch.zeros(b, dtype=torch.uint8, device=DEV)
    if case["aborted"]:
        s["abort"][_aborted(case)] = 1
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = globals()["_prepare_" + case["op"]](case, g)
    s["case"] = case
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

_STATE = ("free_stack", "free_count", "page_tags", "shares", "block_table", "expected_tags")


def _out(s, *more):
    return {name: s[name] for name in _STATE + more}


def _put(into, at, value, where):
    """into[at] = value where `where`; the places are different ones."""
    pad = torch.cat([into, into.new_zeros(1)])
    pad.scatter_(0, torch.where(where, at, into.numel()).long(), value.to(into.dtype))
    into.copy_(pad[:-1])


def _plain_fork(s):
    p = s["case"]["p"]
    src, dst, tok = s["src"].long(), s["dst"].long(), s["tokens"].long()
    table, expected, mp = s["block_table"], s["expected_tags"], s["block_table"].shape[1]
    full, cut = tok // p, tok % p > 0
    nth = torch.cumsum(cut.long(), 0)
    ok = nth <= s["free_count"]
    share = (_columns(mp) < full[:, None]) & ok[:, None]
    theirs = table[src]
    table[dst] = torch.where(share, theirs, table[dst])
    expected[dst] = torch.where(share, expected[src], expected[dst])
    held = torch.zeros(s["shares"].numel() + 1, dtype=torch.int32, device=DEV)
    held.index_add_(0, torch.where(share, theirs, -1).long().flatten() % held.numel(),
                    share.flatten().to(torch.int32))
    s["shares"] += held[:-1]
    new = ok & cut
    page = s["free_stack"][(s["free_count"] - nth).clamp(min=0).long()]
    _put(s["page_tags"], page, s["page_tags"][page.long()] + 1, new)
    place = dst * mp + full
    _put(table.view(-1), place, page, new)
    _put(expected.view(-1), place, s["page_tags"][page.long()], new)
    last = theirs.gather(1, full.clamp(max=mp - 1)[:, None])[:, 0]
    s["copy_src"].copy_(torch.where(new, last, -1))
    s["copy_dst"].copy_(torch.where(new, page, -1))
    s["ok"].copy_(ok)
    s["free_count"] -= new.sum()
    return _out(s, "copy_src", "copy_dst", "ok")


def _plain_release(s):
    table, mp = s["block_table"], s["block_table"].shape[1]
    pages = s["free_stack"].numel()
    req, first, n = s["req"].long(), s["first"].long(), s["npages"].long()
    col = _columns(mp)
    gone = (col >= first[:, None]) & (col < (first + n)[:, None])
    item = torch.where(gone, table[req], pages).long().flatten()  # in list order
    gone = gone.flatten()
    count = torch.zeros(pages + 1, dtype=torch.int64, device=DEV)
    count.index_add_(0, item, torch.ones_like(item))
    nth = torch.arange(item.numel(), device=DEV)
    last = torch.full((pages + 1,), -1, device=DEV).scatter_reduce(0, item, nth, "amax")
    shares = torch.cat([s["shares"], s["shares"].new_zeros(1)])
    freed = gone & (count == shares + 1)[item] & (last[item] == nth)
    _put(s["free_stack"], s["free_count"] + torch.cumsum(freed.long(), 0) - 1, item, freed)
    s["free_count"] += freed.sum()
    s["shares"].copy_((shares - count).clamp(min=0)[:pages])
    table[req] = torch.where(gone.view(-1, mp), -1, table[req])
    return _out(s)


def _plain_compact(s):
    table, expected = s["block_table"], s["expected_tags"]
    n = s["free_stack"].numel()
    page = torch.arange(n, device=DEV)
    free = torch.zeros(n, dtype=torch.bool, device=DEV)
    _put(free, s["free_stack"], torch.ones_like(s["free_stack"]), page < s["free_count"])
    live = n - s["free_count"]
    hole, mover = free & (page < live), ~free & (page >= live)
    holes, movers = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    rank = torch.cumsum(mover.long(), 0) - 1
    _put(holes, torch.cumsum(hole.long(), 0) - 1, page, hole)
    _put(movers, rank, page, mover)
    to = torch.where(mover, holes[rank.clamp(min=0)], page.to(torch.int32))
    tags = s["page_tags"]
    tags += hole.to(torch.int32)
    moved = page < mover.sum()
    s["copy_src"].copy_(torch.where(moved, movers, -1))
    s["copy_dst"].copy_(torch.where(moved, holes, -1))
    s["moves"].copy_(mover.sum())
    shares = s["shares"].clone()
    _put(s["shares"], holes, shares[movers.long()], moved)
    s["shares"].masked_fill_(mover, 0)
    s["free_stack"].copy_(torch.where(page < s["free_count"], n - 1 - page, s["free_stack"]))
    held = _columns(table.shape[1]) < s["held"][:, None]
    at = table.clamp(min=0).long()
    move = held & mover[at]
    table.copy_(torch.where(move, to[at], table))
    expected.copy_(torch.where(move, tags[to[at].long()], expected))
    return _out(s, "copy_src", "copy_dst", "moves")


def _cache_out(s):
    return {name: s[name] for name in ("k_pool", "v_pool", "scales")}


def _plain_copy(s):
    src, dst = s["copy_src"].long(), s["copy_dst"].long()
    for name in ("k_pool", "v_pool"):
        codes = s[name].view(torch.uint8)
        codes[dst] = codes[src]
    s["scales"][dst] = s["scales"][src]
    return _cache_out(s)


def _rows_of(pool, scale, table):
    """The pages of every row of a table one after another: [B, H, MP * P, D] in 32 bits."""
    x = pool.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    x *= scale[table][:, :, :, None, None]
    b, mp, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, mp * p, d)


def _part(s, q, table, hidden):
    """Scores' maximum, sum of weights and weighted values of q [B, n, Hq, D] over the tokens of
    the table's pages that `hidden` [B, n, tokens] leaves; each [B, n, Hq, ...]."""
    b, n, hq, d = q.shape
    h = s["case"]["hkv"]
    g = hq // h
    q = q.float().view(b, n, h, g, d).permute(0, 2, 1, 3, 4).reshape(b, h, n * g, d)
    x = q @ _rows_of(s["k_pool"], s["scales"][:, :, 0], table).transpose(2, 3)
    x *= 1.0 / math.sqrt(d)
    x.view(b, h, n, g, -1).masked_fill_(hidden[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m.clamp(min=-1e30)).exp_()
    o = x @ _rows_of(s["v_pool"], s["scales"][:, :, 1], table)
    return tuple(y.view(b, h, n, g, -1).permute(0, 2, 1, 3, 4).reshape(b, n, hq, -1)
                 for y in (m, x.sum(-1, keepdim=True), o))


def _plain_attn(s):
    case = s["case"]
    b, p, n = case["b"], case["p"], s["n_max"]
    rows, pre_pages, own_pages = s["most"]
    start, lens, table = s["tok_start"].long(), s["seq_lens"].long(), s["block_table"].long()
    at, pre = s["group_start"].long(), s["prefix_pages"].long()
    of = torch.searchsorted(at[1:].contiguous(), torch.arange(b, device=DEV), right=True)
    count = start[1:] - start[:-1]
    most = s["q"].shape[0] - 1
    # the prefixes, for all rows of a group
    r = start[at[:-1], None] + torch.arange(rows, device=DEV)
    hidden = torch.arange(pre_pages * p, device=DEV) >= pre[:, None, None] * p
    one = _part(s, s["q"][r.clamp(max=most)], table[at[:-1], :pre_pages].clamp(min=0),
                hidden.expand(-1, rows, -1))
    # each request's own tokens
    i = torch.arange(n, device=DEV)
    first = pre[of]
    page = (first[:, None] + torch.arange(own_pages, device=DEV)).clamp(max=table.shape[1] - 1)
    sees = (lens - count + 1 - first * p)[:, None] + i
    hidden = torch.arange(own_pages * p, device=DEV) >= sees[:, :, None]
    two = _part(s, s["q"][(start[:-1, None] + i).clamp(max=most)], table.gather(1, page).clamp(min=0),
                hidden)
    # both, by row
    row = torch.arange(s["q"].shape[0], device=DEV)
    req = torch.searchsorted(start[1:].contiguous(), row, right=True)
    live = row < start[-1]  # rows behind the last request stay as they are
    req = req.clamp(max=b - 1)
    one = [x[of[req], (row - start[at[of[req]]]).clamp(0, rows - 1)] for x in one]
    two = [x[req, (row - start[req]).clamp(0, n - 1)] for x in two]
    m = torch.maximum(one[0], two[0])
    e1, e2 = torch.exp(one[0] - m), torch.exp(two[0] - m)
    o = (e1 * one[2] + e2 * two[2]) / (e1 * one[1] + e2 * two[1])
    o = torch.where((s["abort"] != 0)[req, None, None], 0.0, o)
    s["out"].copy_(torch.where(live[:, None, None], o, s["out"].float()))
    return {"out": s["out"]}


# ----------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------

def _handles(s):
    """What a program sets up once beside its buffers."""
    from fp8_paged_kv_attn_gb300 import kvq
    case = s["case"]
    o = {"kvq": kvq}
    if "k_pool" in s:
        o["cache"] = kvq.BlockKVCache(s["k_pool"], s["v_pool"], s["scales"])
    else:
        o["state"] = kvq.PageState(s["free_stack"], s["free_count"], s["page_tags"],
                                   s["block_table"], s["expected_tags"])
        o["ws"] = kvq.pages_workspace(s["free_stack"].shape[0], s["block_table"].shape[0], DEV)
    if case["op"] == "attn":
        o["ws"] = kvq.block_prefix_workspace(s["q"].shape[0], case["hq"], case["hkv"], case["d"], DEV)
    return o


def _own_fork(s, o):
    o["kvq"].kvq_pages_fork(o["state"], s["shares"], s["src"], s["dst"], s["tokens"],
                            s["case"]["p"], s["copy_src"], s["copy_dst"], s["ok"], o["ws"])
    return _out(s, "copy_src", "copy_dst", "ok")


def _own_release(s, o):
    o["kvq"].kvq_pages_release(o["state"], s["shares"], s["req"], s["first"], s["npages"], o["ws"])
    return _out(s)


def _own_compact(s, o):
    o["kvq"].kvq_pages_compact(o["state"], s["shares"], s["held"], s["copy_src"], s["copy_dst"],
                               s["moves"], o["ws"])
    return _out(s, "copy_src", "copy_dst", "moves")


def _own_copy(s, o):
    o["kvq"].kvq_block_copy_pages(o["cache"], s["copy_src"], s["copy_dst"])
    return _cache_out(s)


def _own_attn(s, o):
    o["kvq"].kvq_block_prefix_attn(o["cache"], s["q"], s["tok_start"], s["seq_lens"],
                                   s["block_table"], s["group_start"], s["prefix_pages"], s["out"],
                                   o["ws"], max_q=s["n_max"], abort_mask=s["abort"])
    return {"out": s["out"]}


def run(s):
    op = s["case"]["op"]
    if "live" in s:
        s["live"].copy_(s["saved"])
    if not own:
        return globals()["_plain_" + op](s)
    if "handles" not in s:
        s["handles"] = _handles(s)
    return globals()["_own_" + op](s, s["handles"])


# ----------------------------------------------------------------------------
# the definitions: one request after another, and attention in 64 bits
# ----------------------------------------------------------------------------

def _host(s):
    return {name: s[name].cpu().numpy().copy() for name in _STATE}


def _exact_fork(case, s):
    x, p = _host(s), case["p"]
    count = int(x["free_count"][0])
    n = case["forks"]
    out = {"copy_src": np.full(n, -1, np.int32), "copy_dst": np.full(n, -1, np.int32),
           "ok": np.zeros(n, np.uint8)}
    for i, (a, b, t) in enumerate(zip(*(s[k].tolist() for k in ("src", "dst", "tokens")))):
        full, new = t // p, int(t % p > 0)
        if new > count:
            break
        out["ok"][i] = 1
        for name in ("block_table", "expected_tags"):
            x[name][b, :full] = x[name][a, :full]
        x["shares"][x["block_table"][a, :full]] += 1
        if new:
            count -= 1
            page = x["free_stack"][count]
            x["page_tags"][page] += 1
            x["block_table"][b, full], x["expected_tags"][b, full] = page, x["page_tags"][page]
            out["copy_src"][i], out["copy_dst"][i] = x["block_table"][a, full], page
    x["free_count"][0] = count
    return x | out


def _exact_release(case, s):
    x = _host(s)
    count, shares, stack = int(x["free_count"][0]), x["shares"].tolist(), x["free_stack"]
    for a, f, n in zip(*(s[k].tolist() for k in ("req", "first", "npages"))):
        for page in x["block_table"][a, f:f + n].tolist():
            if shares[page]:
                shares[page] -= 1
            else:
                stack[count] = page
                count += 1
        x["block_table"][a, f:f + n] = -1
    x["free_count"][0] = count
    x["shares"][:] = shares
    return x


def _exact_compact(case, s):
    x = _host(s)
    n, count = case["pages"], int(x["free_count"][0])
    free = np.sort(x["free_stack"][:count])
    live = np.setdiff1d(np.arange(n, dtype=np.int32), free)
    src, dst = live[live >= len(live)], free[free < len(live)]
    out = {"copy_src": np.full(n, -1, np.int32), "copy_dst": np.full(n, -1, np.int32),
           "moves": np.array([len(src)], np.int32)}
    out["copy_src"][:len(src)], out["copy_dst"][:len(src)] = src, dst
    to = np.arange(n, dtype=np.int32)
    to[src] = dst
    x["page_tags"][dst] += 1
    x["shares"][dst], x["shares"][src] = x["shares"][src], 0
    for b, held in enumerate(s["held"].tolist()):
        row = x["block_table"][b, :held]
        moved = to[row] != row
        x["expected_tags"][b, :held][moved] = x["page_tags"][to[row]][moved]
        x["block_table"][b, :held] = to[row]
    x["free_stack"][:count] = np.arange(n - 1, n - 1 - count, -1)
    return x | out


def _exact_copy(case, s):
    src, dst = s["copy_src"].cpu().numpy(), s["copy_dst"].cpu().numpy()
    come = np.arange(case["pages"])
    come[dst] = src
    come = torch.from_numpy(come).to(DEV)
    out = {}
    for name in ("k_pool", "v_pool"):
        out[name] = s[name].view(torch.uint8).index_select(0, come).view(torch.float8_e4m3fn)
    return out | {"scales": s["scales"].index_select(0, come)}


def _exact_attn(case, s):
    n, at, pre, of, total = _attn_plan(case)
    h, p, d = case["hkv"], case["p"], case["d"]
    g = case["hq"] // h
    out = s["out"].double().clone()
    start = np.concatenate([[0], np.cumsum(n)])

    def cached(table):
        x = []
        for i, pool in enumerate((s["k_pool"], s["v_pool"])):
            y = pool.view(torch.uint8).index_select(0, table).view(torch.float8_e4m3fn).double()
            x.append((y * s["scales"][table][:, :, i, None, None].double()).transpose(0, 1).reshape(h, -1, d))
        return x

    for k in range(case["groups"]):
        b0, b1, t = int(at[k]), int(at[k + 1]), int(pre[k])
        first, last = int(start[b0]), int(start[b1])
        q = s["q"][first:last].double().view(last - first, h, g, d) / math.sqrt(d)
        kp, vp = cached(s["block_table"][b0, :t])
        own_kv = [cached(s["block_table"][b, t:-(-int(total[b]) // p)]) for b in range(b0, b1)]
        for head in range(h):
            qh = q[:, head].reshape(-1, d)
            top = torch.full_like(qh[:, :1], -math.inf)
            num, den = torch.zeros_like(qh), torch.zeros_like(top)
            if t:
                x = qh @ kp[head].T
                top = x.amax(-1, keepdim=True)
                x = torch.exp(x - top)
                num, den = x @ vp[head], x.sum(-1, keepdim=True)
            for b in range(b0, b1):
                length, m = int(total[b]) - t * p, int(n[b])
                rows = slice((int(start[b]) - first) * g, (int(start[b + 1]) - first) * g)
                ko, vo = (x[head, :length] for x in own_kv[b - b0])
                x = qh[rows] @ ko.T
                sees = length - m + torch.arange(m, device=DEV).repeat_interleave(g)
                x[torch.arange(length, device=DEV)[None, :] > sees[:, None]] = -math.inf
                high = torch.maximum(top[rows], x.amax(-1, keepdim=True))
                f, x = torch.exp(top[rows] - high), torch.exp(x - high)
                o = (f * num[rows] + x @ vo) / (f * den[rows] + x.sum(-1, keepdim=True))
                out[start[b]:start[b + 1], head * g:(head + 1) * g] = o.view(m, g, d)
    if case["aborted"]:
        b = _aborted(case)
        out[start[b]:start[b + 1]] = 0
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)
