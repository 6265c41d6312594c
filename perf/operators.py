"""Cases of the block-scaled 8-bit cache: rotary positions, quantising the
cache as it is written and reading it back, and attention over it.

Each case is one call that a serving program makes.  ``own`` false computes it
with elementary torch operations, true makes the framework's call.  Requests
are ragged: request b owns rows tok_start[b] .. tok_start[b + 1] - 1 of the
step's tokens, and seq_lens[b] is its length after the step.  K and V lie in
pages of page_size tokens, e4m3 with one power-of-two scale for each (page, kv
head) of K and of V.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -126  # smallest scale exponent (an all-zero block's)


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one decode step's q and k of 64 requests: latency counts
        {"name": "rope_decode_64", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "d": 128,
         "rd": 128, "layout": "half", "scaling": "plain", "far": 9192},
        # prompts with half of each head rotated, frequencies scaled for long contexts
        {"name": "rope_prompt_32k_interleaved", "op": "rope", "tokens": 32768, "hq": 64, "hkv": 8,
         "d": 128, "rd": 64, "layout": "interleaved", "scaling": "ramp", "far": 131072},
        # the decode step of the 64-request sweep point: rotate, quantise, write one token each
        {"name": "append_decode_64_rope", "op": "append", "rope": True, "b": 64, "new_lo": 1,
         "new_hi": 1, "ctx_lo": 8192, "ctx_hi": 9191, "hq": 32, "hkv": 8, "d": 128, "p": 16,
         "rd": 128, "layout": "half", "scaling": "plain", "mix": 1},
        # drafted tokens of many requests, some tokens falling into pages half full
        {"name": "append_draft_256_rope", "op": "append", "rope": True, "b": 256, "new_lo": 1,
         "new_hi": 8, "ctx_lo": 1024, "ctx_hi": 4096, "hq": 32, "hkv": 8, "d": 128, "p": 64,
         "rd": 64, "layout": "interleaved", "scaling": "linear", "mix": 2},
        # whole prompts into the cache: bandwidth
        {"name": "append_prompts_64x8192", "op": "append", "rope": False, "b": 64, "new_lo": 8192,
         "new_hi": 8192, "ctx_lo": 0, "ctx_hi": 0, "hq": 32, "hkv": 8, "d": 128, "p": 16,
         "rd": 128, "layout": "half", "scaling": "plain", "mix": 3},
        # one short prefix read back, of an odd length, small heads
        {"name": "read_one_700", "op": "read", "b": 1, "new_lo": 700, "new_hi": 700, "ctx_lo": 37,
         "ctx_hi": 37, "hkv": 2, "d": 64, "p": 16, "mix": 4},
        # ragged prefixes read back, of 64-token pages
        {"name": "read_prefixes_ragged", "op": "read", "b": 48, "new_lo": 512, "new_hi": 16384,
         "ctx_lo": 0, "ctx_hi": 200, "hkv": 8, "d": 128, "p": 64, "mix": 5},
        # one decode token over 8 requests of 8192 cached tokens
        {"name": "attn_8x8192", "op": "attn", "b": 8, "n_lo": 1, "n_hi": 1, "len_lo": 8193,
         "len_hi": 8193, "hq": 32, "hkv": 8, "d": 128, "p": 16, "pad": 0, "aborted": 0, "mix": 6},
        # the 64-request sweep point
        {"name": "attn_64x9k", "op": "attn", "b": 64, "n_lo": 1, "n_hi": 1, "len_lo": 8193,
         "len_hi": 9192, "hq": 32, "hkv": 8, "d": 128, "p": 16, "pad": 0, "aborted": 0, "mix": 7},
        # lengths from short to long in one batch, 8 query heads a kv head, 64-token pages
        {"name": "attn_ragged_g8_p64", "op": "attn", "b": 64, "n_lo": 1, "n_hi": 1, "len_lo": 512,
         "len_hi": 65536, "hq": 64, "hkv": 8, "d": 128, "p": 64, "pad": 0, "aborted": 0, "mix": 8},
        # a batch of drafted tokens, padded behind the last request
        {"name": "attn_draft_32_n1to8", "op": "attn", "b": 32, "n_lo": 1, "n_hi": 8,
         "len_lo": 1024, "len_hi": 16384, "hq": 32, "hkv": 8, "d": 128, "p": 16, "pad": 19,
         "aborted": 1, "mix": 9},
        # long drafts of a small model: short lengths, odd head counts
        {"name": "attn_draft_d64_n16", "op": "attn", "b": 24, "n_lo": 4, "n_hi": 16, "len_lo": 16,
         "len_hi": 2500, "hq": 18, "hkv": 3, "d": 64, "p": 32, "pad": 5, "aborted": 1, "mix": 10},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attn", "attn"])
    d = rng.choice([64, 128, 128])
    p = rng.choice([16, 32, 64])
    g = rng.choice([1, 2, 3, 4, 4, 6, 8, 8])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    rot = {"rd": rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)]),
           "layout": rng.choice(["half", "interleaved"]),
           "scaling": rng.choice(["plain", "linear", "ramp", "bands"])}
    if op == "rope":
        return {"op": op, "tokens": _log_int(rng, 1, 20000), "hq": g * hkv, "hkv": hkv, "d": d,
                "far": _log_int(rng, 64, 1000000), **rot}
    if op == "append":
        b = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, min(8192, 100000 // b))
        ctx = rng.choice([0, _log_int(rng, 1, 4096)])
        return {"op": op, "rope": rng.random() < 0.6, "b": b, "new_lo": rng.choice([0, 1, hi]),
                "new_hi": hi, "ctx_lo": min(ctx, rng.randint(0, 40)), "ctx_hi": ctx, "hq": g * hkv,
                "hkv": hkv, "d": d, "p": p, "mix": rng.randrange(1 << 20), **rot}
    if op == "read":
        b = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, min(16384, 200000 // b))
        return {"op": op, "b": b, "new_lo": rng.choice([0, 1, hi]), "new_hi": hi, "ctx_lo": 0,
                "ctx_hi": _log_int(rng, 1, 2000), "hkv": hkv, "d": d, "p": p,
                "mix": rng.randrange(1 << 20)}
    b = _log_int(rng, 1, 160)
    hi = _log_int(rng, 16, min(60000, 600000 // b))
    n_hi = rng.choice([1, 1, rng.randint(2, 16)])
    return {"op": op, "b": b, "n_lo": rng.choice([1, n_hi]), "n_hi": n_hi,
            "len_lo": min(hi, max(16, hi // rng.choice([1, 4, 64]))), "len_hi": hi, "hq": g * hkv,
            "hkv": hkv, "d": d, "p": p, "pad": rng.choice([0, rng.randint(1, 9)]),
            "aborted": rng.choice([0, 0, 1]), "mix": rng.randrange(1 << 20)}


def _spread(r, lo, hi, n):
    """n whole numbers of [lo, hi], spread over their logarithm; both ends among them."""
    a = np.exp(r.uniform(np.log(lo + 1), np.log(hi + 1), n)) - 1
    a = np.clip(np.round(a), lo, hi).astype(np.int64)
    if n > 1:
        a[0], a[n - 1] = hi, lo
    return a


def _lengths(case):
    """(tokens of the step, tokens before it) of every request: from the case alone."""
    r = np.random.RandomState(case["mix"])
    b = case["b"]
    if case["op"] == "attn":
        n = r.randint(case["n_lo"], case["n_hi"] + 1, b)
        total = np.maximum(_spread(r, case["len_lo"], case["len_hi"], b), n)
        return n.astype(np.int64), total - n
    n = _spread(r, case["new_lo"], case["new_hi"], b)
    return n, r.randint(case["ctx_lo"], case["ctx_hi"] + 1, b).astype(np.int64)


def _aborted(case):
    """The request that the tag check aborted, if one was."""
    return case["b"] // 2 if case["aborted"] else -1


def work(case):
    if case["op"] == "rope":
        n, h = case["tokens"], case["hq"] + case["hkv"]
        return {"bytes": 4 * n * h * case["d"] + 4 * n + 4 * case["rd"],
                "flops": 3 * n * h * case["rd"]}
    n, ctx = _lengths(case)
    h, d, p = case["hkv"], case["d"], case["p"]
    total = n + ctx
    if case["op"] == "attn":
        live = np.arange(case["b"]) != _aborted(case)
        n, total = n * live, total * live
        pages = int(np.sum(-(-total // p)))
        seen = int(np.sum(n * total - n * (n - 1) // 2))
        return {"bytes": int(total.sum()) * 2 * h * d + pages * (8 * h + 4) +
                int(n.sum()) * case["hq"] * d * 6, "flops": 4 * seen * case["hq"] * d}
    tokens = int(n.sum())
    pages = int(np.sum(np.where(n > 0, -(-total // p) - ctx // p, 0)))
    by = tokens * 2 * h * d * 3 + pages * (8 * h + 4)
    if case["op"] == "append" and case["rope"]:
        by += tokens * case["hq"] * d * 4
    return {"bytes": by, "flops": 2 * tokens * 2 * h * d}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _angles_per_token(case):
    """(radians per position of each pair, factor on the rotated values): plain
    base 10000; positions divided by 8; or frequencies scaled by wavelength,
    with a ramp over pairs or with two bands, for a model trained on 4096."""
    rd, s, trained = case["rd"], 8.0, 4096.0
    i = np.arange(rd // 2, dtype=np.float64)
    f = 10000.0 ** (-2.0 * i / rd)
    if case["scaling"] == "plain":
        return f, 1.0
    if case["scaling"] == "linear":
        return f / s, 1.0
    turns = trained * f / (2 * math.pi)
    if case["scaling"] == "bands":
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f / s * (1 - keep) + f * keep, 1.0
    lo = math.floor(rd * math.log(trained / (32.0 * 2 * math.pi)) / (2 * math.log(10000.0)))
    hi = math.ceil(rd * math.log(trained / (1.0 * 2 * math.pi)) / (2 * math.log(10000.0)))
    lo, hi = max(lo, 0), min(hi, rd - 1)
    keep = 1.0 - np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f / s * (1 - keep) + f * keep, 0.1 * math.log(s) + 1.0


def _values(g, shape):
    """bf16 activations: heads of different size, some large values."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-3, 4, (shape[-2], 1), generator=g, device="cuda").float())
    x *= torch.where(torch.rand(shape[-1], generator=g, device="cuda") < 0.02, 12.0, 1.0)
    return x.to(torch.bfloat16)


def _pool(g, pages, h, p, d):
    """A pool as a run of the cache leaves it: codes and scales of random pages."""
    codes = torch.empty(pages, h, p, d, dtype=torch.uint8, device="cuda")
    exp = torch.empty(pages, h, device="cuda")
    step = max(1, (1 << 27) // (h * p * d))
    for at in range(0, pages, step):
        x = torch.randn(min(step, pages - at), h, p, d, generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-3, 4, (x.shape[0], h, 1, 1), generator=g,
                                      device="cuda").float())
        e = torch.ceil(torch.log2(x.abs().amax((2, 3)) / E4M3_MAX))
        codes[at:at + step] = (x * torch.exp2(-e)[:, :, None, None]).clamp_(-448, 448) \
            .to(torch.float8_e4m3fn).view(torch.uint8)
        exp[at:at + step] = e
    return codes.view(torch.float8_e4m3fn), torch.exp2(exp)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rope" or case.get("rope"):
        f, s["mscale"] = _angles_per_token(case)
        s["inv_freq"] = torch.from_numpy(f).cuda()
    d = case["d"]
    if case["op"] == "rope":
        n = case["tokens"]
        s["q"], s["k"] = _values(g, (n, case["hq"], d)), _values(g, (n, case["hkv"], d))
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["pos"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda",
                                 dtype=torch.int32)
        return s
    h, p, b = case["hkv"], case["p"], case["b"]
    n, ctx = _lengths(case)
    total = n + ctx
    mp = max(1, int(-(-total.max() // p)))
    used = -(-total // p)
    pages = max(1, int(used.sum() * 1.05) + 1)
    table = torch.full((b, mp), -1, dtype=torch.int32, device="cuda")
    mine = torch.arange(mp, device="cuda")[None, :] < torch.from_numpy(used).cuda()[:, None]
    table[mine] = torch.randperm(pages, generator=g, device="cuda")[:int(used.sum())].to(torch.int32)
    s["block_table"] = table
    start = np.concatenate([[0], np.cumsum(n)])
    s["tok_start"] = torch.from_numpy(start).to(torch.int32).cuda()
    s["seq_lens"] = torch.from_numpy(total).to(torch.int32).cuda()
    s["k_pool"], ks = _pool(g, pages, h, p, d)
    s["v_pool"], vs = _pool(g, pages, h, p, d)
    s["scales"] = torch.stack([ks, vs], dim=2).contiguous()
    rows = int(start[-1])
    if case["op"] == "append":
        s["into"] = torch.from_numpy(np.nonzero((n > 0) & (ctx % p > 0))[0]).cuda()
        s["k"], s["v"] = _values(g, (rows, h, d)), _values(g, (rows, h, d))
        if case["rope"]:
            s["q"] = _values(g, (rows, case["hq"], d))
            s["q_out"] = torch.empty_like(s["q"])
    elif case["op"] == "read":
        s["first"] = torch.from_numpy(ctx).to(torch.int32).cuda()
        s["k_out"] = torch.zeros(rows, h, d, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        rows += case["pad"]
        s["q"] = _values(g, (rows, case["hq"], d))
        s["out"] = torch.zeros(rows, case["hq"], d, device="cuda")
        s["n_max"] = int(n.max())
        s["abort"] = torch.zeros(b, dtype=torch.uint8, device="cuda")
        if case["aborted"]:
            s["abort"][_aborted(case)] = 1
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _rotated(x, pos, s):
    """x [N, H, D] in 32 bits with its first rotary_dim dims rotated; angles in 64."""
    case = s["case"]
    rd = case["rd"]
    t = pos.double()[:, None] * s["inv_freq"][None, :]
    c = (t.cos() * s["mscale"]).float()[:, None, :]
    i = (t.sin() * s["mscale"]).float()[:, None, :]
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., :rd // 2], y[..., rd // 2:rd]
        return torch.cat([a * c - b * i, b * c + a * i, y[..., rd:]], -1)
    a, b = y[..., 0:rd:2], y[..., 1:rd:2]
    return torch.cat([torch.stack([a * c - b * i, b * c + a * i], -1).flatten(-2), y[..., rd:]], -1)


def _owners(s, rows):
    """Request and position of each of the step's rows."""
    start = s["tok_start"].long()
    row = torch.arange(rows, device="cuda")
    req = torch.searchsorted(start[1:].contiguous(), row, right=True)
    return req, row, start


def _block_scale(amax):
    """The smallest power of two s with amax / s <= 448 = 0.875 2^9."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, MIN_EXP).clamp(min=MIN_EXP)
    return torch.exp2(e.float())


def _codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _write(pool, scales, x, page, slot, old_page, old_n):
    """Quantise x [N, H, D] into pool; the pages of old_page hold old_n tokens already."""
    need = _block_scale(torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax"))
    was = torch.zeros_like(scales)
    was[old_page] = scales[old_page]
    new = torch.maximum(need, was)
    codes = pool.view(torch.uint8)
    kept = pool[old_page].float() * (scales[old_page] / new[old_page])[:, :, None, None]
    is_old = torch.arange(pool.shape[2], device="cuda")[None, :] < old_n[:, None]
    codes[old_page] = torch.where(is_old[:, None, :, None], _codes(kept), codes[old_page])
    codes[page, :, slot] = _codes(x / new[page][:, :, None])
    scales[page] = new[page]


def _plain_append(s):
    case = s["case"]
    p = case["p"]
    req, row, start = _owners(s, s["k"].shape[0])
    lens, table = s["seq_lens"].long(), s["block_table"].long()
    pos = lens[req] - start[req + 1] + row
    k = s["k"].float()
    if case["rope"]:
        s["q_out"].copy_(_rotated(s["q"], pos, s))
        k = _rotated(s["k"], pos, s)
    page, slot = table[req, pos // p], pos % p
    into = s["into"]  # requests whose first new token falls into a page with tokens
    before = lens[into] - (start[into + 1] - start[into])
    old_page, old_n = table[into, before // p], before % p
    for i, (pool, x) in enumerate(((s["k_pool"], k), (s["v_pool"], s["v"].float()))):
        plane = s["scales"][:, :, i].contiguous()
        _write(pool, plane, x, page, slot, old_page, old_n)
        s["scales"][:, :, i] = plane
    return _cache_out(s)


def _cache_out(s):
    out = {"k_pool": s["k_pool"], "v_pool": s["v_pool"], "scales": s["scales"]}
    return out | ({"q": s["q_out"]} if s["case"]["rope"] else {})


def _plain_rope(s):
    s["q_out"].copy_(_rotated(s["q"], s["pos"], s))
    s["k_out"].copy_(_rotated(s["k"], s["pos"], s))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_read(s):
    p = s["case"]["p"]
    req, row, start = _owners(s, s["k_out"].shape[0])
    pos = s["first"].long()[req] + row - start[req]
    page, slot = s["block_table"].long()[req, pos // p], pos % p
    for i, (pool, to) in enumerate(((s["k_pool"], s["k_out"]), (s["v_pool"], s["v_out"]))):
        to.copy_(pool.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float() *
                 s["scales"][page, :, i][:, :, None])
    return {"k": s["k_out"], "v": s["v_out"]}


def _padded(pool, scale, table):
    """Every request's pages one after another: [B, H, MP * P, D] in 32 bits."""
    x = pool.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    x *= scale[table][:, :, :, None, None]
    b, mp, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, mp * p, d)


def _plain_attn(s):
    case = s["case"]
    b, h, d, n = case["b"], case["hkv"], case["d"], s["n_max"]
    g = case["hq"] // h
    start, lens = s["tok_start"].long(), s["seq_lens"].long()
    count = start[1:] - start[:-1]
    table = s["block_table"].long().clamp(min=0)
    i = torch.arange(n, device="cuda")
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(b, n, h, g, d).permute(0, 2, 1, 3, 4).reshape(b, h, n * g, d)
    x = q @ _padded(s["k_pool"], s["scales"][:, :, 0], table).transpose(2, 3)
    x *= 1.0 / math.sqrt(d)
    seen = lens[:, None] - count[:, None] + 1 + i  # keys that query i of each request sees
    hidden = torch.arange(x.shape[-1], device="cuda") >= seen[:, :, None]
    x.view(b, h, n, g, -1).masked_fill_(hidden[:, None, :, None, :], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = (x @ _padded(s["v_pool"], s["scales"][:, :, 1], table)) / x.sum(-1, keepdim=True)
    o = o.view(b, h, n, g, d).permute(0, 2, 1, 3, 4).reshape(b, n, h * g, d)
    o = torch.where((s["abort"] != 0)[:, None, None, None], 0.0, o)
    req, at, _ = _owners(s, s["q"].shape[0])
    live = at < start[-1]  # rows behind the last request stay as they are
    req = req.clamp(max=b - 1)
    s["out"].copy_(torch.where(live[:, None, None], o[req, (at - start[req]).clamp(0, n - 1)],
                               s["out"]))
    return {"out": s["out"]}


# ----------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------

def _handles(s):
    """What a program sets up once beside its buffers: the cache's and the
    rotation's descriptions and the attention's workspace."""
    from fp8_paged_kv_attn_gb300 import kvq
    case = s["case"]
    own_ = {"kvq": kvq}
    if "inv_freq" in s:
        layout = kvq.ROPE_HALF if case["layout"] == "half" else kvq.ROPE_INTERLEAVED
        own_["rope"] = kvq.Rope(s["inv_freq"], layout, s["mscale"])
    if "k_pool" in s:
        own_["cache"] = kvq.BlockKVCache(s["k_pool"], s["v_pool"], s["scales"])
    if "n_max" in s:
        own_["ws"] = kvq.block_workspace(case["b"], s["n_max"], case["hq"], case["hkv"],
                                         case["d"])
    return own_


def _own_rope(s, o):
    o["kvq"].kvq_rope(o["rope"], s["pos"], s["q"], s["q_out"], s["k"], s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_append(s, o):
    where = (s["tok_start"], s["seq_lens"], s["block_table"])
    if "rope" in o:
        o["kvq"].kvq_rope_block_append(o["cache"], o["rope"], s["q"], s["q_out"], s["k"], s["v"],
                                       *where)
    else:
        o["kvq"].kvq_block_append(o["cache"], s["k"], s["v"], *where)
    return _cache_out(s)


def _own_read(s, o):
    o["kvq"].kvq_block_read(o["cache"], s["tok_start"], s["first"], s["block_table"], s["k_out"],
                            s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attn(s, o):
    o["kvq"].kvq_block_attn(o["cache"], s["q"], s["tok_start"], s["seq_lens"], s["block_table"],
                            s["out"], o["ws"], max_q=s["n_max"], abort_mask=s["abort"])
    return {"out": s["out"]}


_PLAIN = {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "attn": _plain_attn}
_OWN = {"rope": _own_rope, "append": _own_append, "read": _own_read, "attn": _own_attn}


def run(s):
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    if "handles" not in s:
        s["handles"] = _handles(s)
    return _OWN[op](s, s["handles"])


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

def _exact_rotate(x, pos, case):
    f, m = _angles_per_token(case)
    rd = case["rd"]
    t = torch.outer(pos.double(), torch.from_numpy(f).cuda())
    z = m * torch.polar(torch.ones_like(t), t)[:, None, :]
    y = x.double().clone()
    first = slice(0, rd // 2) if case["layout"] == "half" else slice(0, rd, 2)
    second = slice(rd // 2, rd) if case["layout"] == "half" else slice(1, rd, 2)
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _exact_append(case, s):
    n, ctx = _lengths(case)
    p, h = case["p"], case["hkv"]
    start = np.concatenate([[0], np.cumsum(n)])
    pos = torch.from_numpy(np.concatenate([np.arange(c, c + m) for c, m in zip(ctx, n)])).cuda()
    req = np.repeat(np.arange(case["b"]), n)
    new = {"k_pool": s["k"].double(), "v_pool": s["v"].double()}
    out = {}
    if case["rope"]:
        new["k_pool"] = _exact_rotate(s["k"], pos, case)
        out["q"] = _exact_rotate(s["q"], pos, case)
    page = s["block_table"].cpu().long()[torch.from_numpy(req), (pos // p).cpu()].cuda()
    # tokens that were in a page before: a mask over the pool
    kept = torch.zeros(s["k_pool"].shape[0], p, dtype=torch.bool, device="cuda")
    table = s["block_table"].cpu().numpy()
    into = [b for b in range(case["b"]) if n[b] > 0 and ctx[b] % p]
    if into:
        at = torch.tensor([int(table[b, ctx[b] // p]) for b in into], device="cuda")
        kept[at] = torch.arange(p, device="cuda")[None, :] <             torch.tensor([int(ctx[b] % p) for b in into], device="cuda")[:, None]
    scales = s["scales"].double().clone()
    for i, name in enumerate(("k_pool", "v_pool")):
        pool, x = s[name].double(), new[name]
        amax = torch.zeros(pool.shape[0], h, dtype=torch.float64, device="cuda")
        amax.scatter_reduce_(0, page[:, None].expand(-1, h), x.abs().amax(-1), "amax")
        need = torch.exp2(torch.floor(torch.log2(amax)).clamp(min=MIN_EXP + 8) - 8)
        need = torch.where(amax > E4M3_MAX * need, 2 * need, need)
        had = kept.any(1)[:, None]
        want = torch.where(had, torch.maximum(need, scales[:, :, i]), need)
        touched = torch.zeros(pool.shape[0], dtype=torch.bool, device="cuda")
        touched[page] = True
        if into:
            pool[at] = torch.where(kept[at][:, None, :, None],
                                   pool[at] * (scales[at, :, i] / want[at])[:, :, None, None],
                                   pool[at])
        pool[page, :, pos % p] = (x / want[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        scales[:, :, i] = torch.where(touched[:, None], want, scales[:, :, i])
        out[name] = pool
    return out | {"scales": scales}


def _exact_read(case, s):
    n, ctx = _lengths(case)
    p = case["p"]
    out = {"k": [], "v": []}
    for b in range(case["b"]):
        at = torch.arange(int(ctx[b]), int(ctx[b] + n[b]), device="cuda")
        page = s["block_table"][b].long()[at // p]
        for i, name in enumerate(("k", "v")):
            x = s[name + "_pool"].view(torch.uint8)[page, :, at % p].view(torch.float8_e4m3fn)
            out[name].append(x.double() * s["scales"][page, :, i].double()[:, :, None])
    return {name: torch.cat(x) for name, x in out.items()}


def _exact_attn(case, s):
    n, ctx = _lengths(case)
    p, h, d = case["p"], case["hkv"], case["d"]
    g = case["hq"] // h
    out = s["out"].double().clone()
    row = 0
    for b in range(case["b"]):
        m, total = int(n[b]), int(n[b] + ctx[b])
        if b != _aborted(case):
            pages = s["block_table"][b, :-(-total // p)].long()
            k, v = ((x.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() *
                     s["scales"][pages, :, i].double()[:, :, None, None])
                    .transpose(0, 1).reshape(h, -1, d)[:, :total]
                    for i, x in enumerate((s["k_pool"], s["v_pool"])))
            q = s["q"][row:row + m].double().view(m, h, g, d).permute(1, 0, 2, 3).reshape(h, m * g, d)
            x = q @ k.transpose(1, 2) / math.sqrt(d)
            last = total - m + torch.arange(m, device="cuda").repeat_interleave(g)
            x[:, torch.arange(total, device="cuda")[None, :] > last[:, None]] = -math.inf
            o = torch.softmax(x, -1) @ v
            out[row:row + m] = o.view(h, m, g, d).permute(1, 0, 2, 3).reshape(m, h * g, d)
        row += m
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _exact_rotate(s["q"], s["pos"], case), "k": _exact_rotate(s["k"], s["pos"], case)}
    return globals()["_exact_" + case["op"]](case, s)
