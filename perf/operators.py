"""The operators between a decoder block's LoRA projections, as cases to measure.

Four operators of a paged multi-adapter decode step:

- ``maps``    block tables and slot maps of a batch, from the requests' lengths
- ``append``  new tokens' keys and values written to a cache held in 4 bits (and read back)
- ``attend``  attention of ragged queries over that cache, causal from each request's end
- ``norm``    root-mean-square norm of x + residual, optionally with an e4m3 copy and row scales

``run`` computes them in plain torch operations in 32 bits; with ``own`` set it makes the calls of
``segmented_rank_gemm_gb300.kv`` and ``segmented_rank_gemm_gb300.norm``.

The 4-bit format: 16 consecutive dimensions of one token and head share one scale
s = e4m3(max|x| / (7 g)), g a constant of the cache; codes are round(x / (s g)) in -7..7, kept
with 8 added, and stand for code * s * g.
"""
import random

import numpy as np
import torch

own = False

GROUP = 16
DEV = "cuda"

# The head layout is that of the 8B-class block of this repository's stack: a 4096-wide query
# projection and 1024-wide key and value projections, as 32 and 8 heads of 128.
HEADS = {"hq": 32, "hkv": 8, "d": 128, "page": 64}


def listed():
    return [
        # one step of the stack's decode batch: 512 requests, one token each
        {"name": "maps_decode_512", "op": "maps", "requests": 512, "prompts": 0, "chunk": 1,
         "ctx": 2048, "page": 64},
        # the mixed continuous batch: 8 prompts of 448 tokens beside 512 single tokens
        {"name": "maps_mixed_4096", "op": "maps", "requests": 520, "prompts": 8, "chunk": 448,
         "ctx": 4096, "page": 16},
        # many ragged requests, some idle, and padding at the token arrays' end
        {"name": "maps_ragged_2999", "op": "maps", "requests": 2999, "prompts": 2900, "chunk": 21,
         "ctx": 8192, "page": 32},
        # a decode step's new keys and values
        {"name": "append_512", "op": "append", "tokens": 512, "hkv": 8, "d": 128, "page": 64},
        # a prompt batch's, at the prefill workload's token count, with padding rows
        {"name": "append_8192", "op": "append", "tokens": 8192, "hkv": 8, "d": 128, "page": 64},
        # a single user's next token: the smallest call
        {"name": "attend_one", "op": "attend", "prompts": 0, "chunk": 1, "decodes": 1,
         "ctx": 1000, **HEADS},
        # the stack's decode batch over contexts of very different lengths
        {"name": "attend_decode_512", "op": "attend", "prompts": 0, "chunk": 1, "decodes": 512,
         "ctx": 2048, **HEADS},
        # a few long documents, one token each
        {"name": "attend_long", "op": "attend", "prompts": 0, "chunk": 1, "decodes": 3,
         "ctx": 131072, **HEADS},
        # prompt chunks behind a context that is already cached
        {"name": "attend_prompts", "op": "attend", "prompts": 8, "chunk": 1024, "decodes": 0,
         "ctx": 2048, **HEADS},
        # prompts and single tokens in one batch, small pages
        {"name": "attend_mixed", "op": "attend", "prompts": 8, "chunk": 448, "decodes": 512,
         "ctx": 1024, "hq": 32, "hkv": 8, "d": 128, "page": 16},
        # the decode batch's norm, feeding e4m3 projections
        {"name": "norm_512_e4m3", "op": "norm", "tokens": 512, "k": 4096, "dtype": "bf16",
         "e4m3": True, "residual": True, "pad": 0},
        # the prefill batch's
        {"name": "norm_8192", "op": "norm", "tokens": 8192, "k": 4096, "dtype": "bf16",
         "e4m3": True, "residual": True, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("maps", "append", "attend", "attend", "norm"))
    if op == "maps":
        b = _log_int(rng, 1, 3000)
        return {"op": op, "requests": b, "prompts": rng.randint(0, min(b, 60000 // 448)),
                "chunk": _log_int(rng, 2, 448), "ctx": _log_int(rng, 32, 8192),
                "page": rng.choice((16, 32, 64, 128))}
    heads = {"hkv": rng.choice((1, 2, 3, 4, 8)), "d": rng.choice((64, 128)),
             "page": rng.choice((16, 32, 64, 128))}
    if op == "append":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), **heads}
    if op == "norm":
        e4m3 = rng.random() < 0.5
        return {"op": op, "tokens": _log_int(rng, 1, 8192),
                "k": rng.choice((1024, 4096, 4096 - 8, 2056, rng.randint(65, 4096))),
                "dtype": "bf16" if e4m3 or rng.random() < 0.7 else "f32", "e4m3": e4m3,
                "residual": rng.random() < 0.8, "pad": rng.choice((0, 0, 8, 5))}
    heads["hq"] = heads["hkv"] * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * heads["hkv"] <= 32])
    kind = rng.choice(("decodes", "decodes", "long", "few", "prompts", "mixed"))
    if kind == "decodes":
        n = _log_int(rng, 1, 512)
        return {"op": op, "prompts": 0, "chunk": 1, "decodes": n,
                "ctx": _log_int(rng, 16, 2048), **heads}
    if kind == "long":
        return {"op": op, "prompts": 0, "chunk": 1, "decodes": rng.randint(1, 3),
                "ctx": _log_int(rng, 2048, 100000), **heads}
    if kind == "few":  # several tokens a request: a draft to verify
        return {"op": op, "prompts": _log_int(rng, 1, 64), "chunk": rng.randint(2, 8),
                "decodes": 0, "ctx": _log_int(rng, 16, 2048), **heads}
    chunk = _log_int(rng, 9, 700)
    return {"op": op, "prompts": rng.randint(1, 8), "chunk": chunk,
            "decodes": rng.randint(1, 256) if kind == "mixed" else 0,
            "ctx": chunk + _log_int(rng, 1, 1300), **heads}


# ----------------------------------------------------------------------------------------
# lengths: a function of the case alone, so that work() is exact
# ----------------------------------------------------------------------------------------

def _lengths(case):
    """(cached tokens before the batch, new tokens) of each request; prompts come first."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens, new = [], []
    n_dec = case["requests"] - case["prompts"] if case["op"] == "maps" else case["decodes"]
    for i in range(case["prompts"]):
        n = rng.randint(max(1, case["chunk"] // 2), case["chunk"])
        if case["op"] == "maps" and rng.random() < 0.05:
            n = 0  # an idle request keeps its place in the table
        if i == 0:
            n = case["chunk"]
        new.append(min(n, case["ctx"]))
        lens.append(0 if rng.random() < 0.25 else rng.randint(0, max(0, case["ctx"] - new[-1])))
    for i in range(n_dec):
        new.append(1)
        long = case["ctx"] >= 8192 and case["op"] == "attend"
        lens.append((rng.randint(case["ctx"] // 2, case["ctx"]) if long
                     else _log_int(rng, 1, case["ctx"]) if i else case["ctx"]) - 1)
    return lens, new


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "norm":
        n, size = case["tokens"] * case["k"], 2 if case["dtype"] == "bf16" else 4
        rows = n * size * (2 + 2 * case["residual"])  # x and y; the residual in and out
        return {"bytes": rows + case["k"] * size + (n + 4 * case["tokens"] if case["e4m3"] else 0),
                "flops": 8 * n}
    if case["op"] == "append":
        n = 2 * case["tokens"] * case["hkv"] * case["d"]
        # k and v in, codes and scales written, values read back from them
        return {"bytes": n * 2 + n // 2 + n // GROUP + n * 2 + 4 * case["tokens"], "flops": 4 * n}
    lens, new = _lengths(case)
    if case["op"] == "maps":
        taken = sum(_cdiv(a + b, case["page"]) - _cdiv(a, case["page"]) for a, b in zip(lens, new))
        return {"bytes": 4 * (len(lens) * 5 + 2 * taken + 3 * sum(new)), "flops": sum(new)}
    kv = sum(a + b for a, b in zip(lens, new))
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(lens, new))
    cache = kv * case["hkv"] * case["d"] * 2 * (0.5 + 1 / GROUP)
    return {"bytes": int(cache) + 2 * 2 * sum(new) * case["hq"] * case["d"],
            "flops": 4 * pairs * case["hq"] * case["d"]}


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _keys_values(g, tokens, hkv, d):
    """Keys with channels of very different size, as projections give them, and plain values."""
    size = torch.exp(0.7 * torch.randn(hkv, d, generator=g, device=DEV))
    k = (torch.randn(tokens, hkv, d, generator=g, device=DEV) * size).bfloat16()
    v = (torch.randn(tokens, hkv, d, generator=g, device=DEV) * 0.5).bfloat16()
    return k, v


def _scattered(g, lens, page, spare=3):
    """A block table over shuffled pages: [B, blocks], and the number of pages."""
    blocks = [_cdiv(n, page) for n in lens]
    pages = sum(blocks) + spare
    order = torch.randperm(pages, generator=g, device=DEV).int()
    wide = max(max(blocks), 1)
    start = np.concatenate(([0], np.cumsum(blocks)))[:-1]
    col = np.arange(wide)[None, :]
    at = np.where(col < np.asarray(blocks)[:, None], start[:, None] + col, pages - 1)
    return order[torch.from_numpy(at).to(DEV)].contiguous(), pages


def _slots_of(table, lens, page):
    """The cache slots of tokens 0 .. lens[b]-1 of each request, in order."""
    n = torch.tensor(lens, device=DEV)
    req = torch.repeat_interleave(torch.arange(len(lens), device=DEV), n)
    first = torch.cumsum(n, 0) - n
    pos = torch.arange(int(n.sum()), device=DEV) - first[req]
    return (table[req, pos // page].long() * page + pos % page).int()


def _case_kv(case, seed):
    """Everything of an attend case before the cache is filled."""
    g = _gen(seed)
    lens, new = _lengths(case)
    kv = [a + b for a, b in zip(lens, new)]
    table, pages = _scattered(g, kv, case["page"])
    k, v = _keys_values(g, sum(kv), case["hkv"], case["d"])
    q = torch.randn(sum(new), case["hq"], case["d"], generator=g, device=DEV).bfloat16()
    return {"lens": lens, "new": new, "kv": kv, "table": table, "pages": pages, "k": k, "v": v,
            "q": q, "slots": _slots_of(table, kv, case["page"])}


def _pool(pages, case):
    """An empty plain cache; one row more than its slots takes what padding rows write."""
    rows, h, d = pages * case["page"] + 1, case["hkv"], case["d"]
    return {"kc": torch.zeros(rows, h, d // 2, dtype=torch.uint8, device=DEV),
            "vc": torch.zeros(rows, h, d // 2, dtype=torch.uint8, device=DEV),
            "ks": torch.zeros(rows, h, d // GROUP, device=DEV).to(torch.float8_e4m3fn),
            "vs": torch.zeros(rows, h, d // GROUP, device=DEV).to(torch.float8_e4m3fn)}


def _own_cache(pages, case, requests):
    from segmented_rank_gemm_gb300.kv import KvCache
    return KvCache(pages, case["page"], case["hkv"], case["d"], max_requests=requests)


def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "norm":
        g = _gen(seed)
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        t, k = case["tokens"], case["k"]

        def rows(spread):
            full = torch.randn(t, k + case["pad"], generator=g, device=DEV) * spread
            return full.to(dt)[:, :k]

        st["x"] = rows(1.0)
        st["residual"] = rows(4.0) if case["residual"] else None
        st["weight"] = (1 + 0.1 * torch.randn(k, generator=g, device=DEV)).to(dt)
        st["y"] = torch.empty(t, k, dtype=dt, device=DEV)
        st["h"] = torch.empty(t, k, dtype=dt, device=DEV) if case["residual"] else None
        st["xq"] = st["sx"] = None
        if case["e4m3"]:
            st["xq"] = torch.empty(t, k, dtype=torch.float8_e4m3fn, device=DEV)
            st["sx"] = torch.empty(t, device=DEV)
        return st
    if case["op"] == "maps":
        g = _gen(seed)
        lens, new = _lengths(case)
        page, b = case["page"], len(lens)
        st["table"], used = _scattered(g, lens, page, spare=0)
        more = sum(_cdiv(a + n, page) - _cdiv(a, page) for a, n in zip(lens, new))
        blocks = _cdiv(case["ctx"] + case["chunk"], page)
        wide = torch.zeros(b, blocks, dtype=torch.int32, device=DEV)
        wide[:, :st["table"].shape[1]] = st["table"][:, :blocks]
        tokens = sum(new) + 7  # a captured step pads its token arrays
        st.update(table=wide, tokens=tokens, lens=_ints(lens), new=_ints(new),
                  adapter=torch.randint(-1, 100, (b,), generator=g, device=DEV).int(),
                  free=(used + torch.randperm(more + 64, generator=g, device=DEV)).int(),
                  n_free=_ints([more + 50]))
        for name, n in (("kv_len", b), ("q_offsets", b + 1), ("position", tokens),
                        ("kv_slot", tokens), ("token_slot", tokens), ("counts", 5)):
            st[name] = torch.zeros(n, dtype=torch.int32, device=DEV)
        return st
    if case["op"] == "append":
        g = _gen(seed)
        t, page = case["tokens"], case["page"]
        pages = _cdiv(t, page) * 2 + 1
        st["k"], st["v"] = _keys_values(g, t, case["hkv"], case["d"])
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:t].int()
        slots[t - t // 100:] = -1  # padding rows
        st["slots"] = slots
        if own:
            st["cache"] = _own_cache(pages, case, 1)
        else:
            st["pool"] = _pool(pages, case)
        st["k_out"], st["v_out"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        return st
    d = _case_kv(case, seed)
    st.update(q=d["q"], table=d["table"], kv_len=_ints(d["kv"]), max_q=max(d["new"]),
              q_offsets=_ints(np.concatenate(([0], np.cumsum(d["new"]))).tolist()),
              max_kv=max(d["kv"]), prompt_tokens=sum(d["new"][:case["prompts"]]),
              out=torch.empty_like(d["q"]))
    if own:
        st["cache"] = _own_cache(d["pages"], case, len(d["kv"]))
        st["cache"].append(d["k"], d["v"], d["slots"])
    else:
        st["pool"] = _pool(d["pages"], case)
        _append(st["pool"], d["k"], d["v"], d["slots"])
    return st


# ----------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------

def _over(x, n):
    """x / n, correctly rounded (a division by a Python number multiplies by its reciprocal,
    which turns quotients halfway between two e4m3 values to one side)."""
    return x / torch.full_like(x, n)


def _quantize(x):
    """bf16 [T, H, D] -> packed codes [T, H, D/2] and e4m3 scales [T, H, D/16]."""
    x = x.float().unflatten(-1, (-1, GROUP))
    s = _over(x.abs().amax(-1), 7.0).clamp(max=448).to(torch.float8_e4m3fn)
    f = s.float().unsqueeze(-1)
    code = torch.where(f > 0, torch.round(x / f).clamp(-7, 7), 0.0)
    code = (code.flatten(-2) + 8).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _values(code, s):
    """The 32-bit values of packed codes and their scales."""
    pair = torch.stack((code & 15, code >> 4), -1).flatten(-2)
    x = (pair.float() - 8).unflatten(-1, (-1, GROUP))
    return (x * s.float().unsqueeze(-1)).flatten(-2)


def _append(pool, k, v, slots):
    at = torch.where(slots >= 0, slots, pool["kc"].shape[0] - 1).long()
    pool["kc"][at], ks = _quantize(k)
    pool["vc"][at], vs = _quantize(v)
    pool["ks"].view(torch.uint8)[at] = ks.view(torch.uint8)
    pool["vs"].view(torch.uint8)[at] = vs.view(torch.uint8)


def _rows(codes, scales, at):
    return _values(codes[at], scales.view(torch.uint8)[at].view(torch.float8_e4m3fn))


def _run_append(st):
    pool, slots = st["pool"], st["slots"]
    _append(pool, st["k"], st["v"], slots)
    at = slots.clamp(min=0).long()
    there = (slots >= 0)[:, None, None]
    return [torch.where(there, _rows(pool[c], pool[s], at), 0.0).bfloat16()
            for c, s in (("kc", "ks"), ("vc", "vs"))]


def _attend_part(st, b0, b1, max_q, t0, t1):
    """Requests b0 .. b1-1, whose tokens are t0 .. t1-1, padded to the longest."""
    case, pool = st["case"], st["pool"]
    page, hkv, d = case["page"], case["hkv"], case["d"]
    group = case["hq"] // hkv
    n = b1 - b0
    kv_len, first = st["kv_len"][b0:b1].long(), st["q_offsets"][b0:b1].long()
    q_len = st["q_offsets"][b0 + 1:b1 + 1].long() - first
    pos = torch.arange(st["max_kv"], device=DEV)
    slot = st["table"][b0:b1].long()[:, pos // page] * page + pos % page
    k = _rows(pool["kc"], pool["ks"], slot).permute(0, 2, 3, 1)  # [n, hkv, d, L]
    v = _rows(pool["vc"], pool["vs"], slot).permute(0, 2, 1, 3)  # [n, hkv, L, d]
    i = torch.arange(max_q, device=DEV)
    q = st["q"][(first[:, None] + i).clamp(max=t1 - 1)].float()  # [n, max_q, hq, d]
    q = q.view(n, max_q, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * max_q, d)
    s = torch.matmul(q, k) * d ** -0.5
    last = kv_len[:, None] - q_len[:, None] + i  # the last key a query sees
    seen = pos <= last[:, :, None]  # [n, max_q, L]
    s = s.view(n, hkv, group, max_q, -1).masked_fill(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1)
    o = torch.matmul(p.view(n, hkv, group * max_q, -1), v).view(n, hkv, group, max_q, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, max_q, case["hq"], d)
    token = torch.arange(t0, t1, device=DEV)
    b = torch.searchsorted(first + q_len, token, right=True)
    return o[b, token - first[b]].bfloat16()


def _run_attend(st):
    case = st["case"]
    n, t = case["prompts"], st["q"].shape[0]
    parts = []
    if n:
        parts.append(_attend_part(st, 0, n, case["chunk"], 0, st["prompt_tokens"]))
    if case["decodes"]:
        parts.append(_attend_part(st, n, n + case["decodes"], 1, st["prompt_tokens"], t))
    return torch.cat(parts)


def _run_maps(st):
    page, lens, new, table = st["case"]["page"], st["lens"].long(), st["new"].long(), st["table"]
    end = lens + new
    have, need = (lens + page - 1) // page, (end + page - 1) // page
    taken = torch.cumsum(need - have, 0)
    offsets = torch.cat((torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)))
    total, pages, n_free = offsets[-1], taken[-1], st["n_free"][0].long()
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    which = n_free - 1 - (taken - (need - have))[:, None] - (col - have[:, None])
    fresh = (col >= have[:, None]) & (col < need[:, None])
    table = torch.where(fresh, st["free"][which.clamp(0, st["free"].shape[0] - 1)], table)
    token = torch.arange(st["tokens"], device=DEV)
    r = torch.searchsorted(offsets[1:], token, right=True).clamp(max=lens.shape[0] - 1)
    there = token < total
    pos = lens[r] + token - offsets[r]
    pos = torch.where(there, pos, 0)
    slot = torch.where(there, table[r, pos // page] * page + pos % page, -1)
    adapter = torch.where(there, st["adapter"][r], -1)
    counts = torch.stack((total, n_free - pages, pages))
    return [x.int() for x in (table, end, offsets, pos, slot, adapter, counts)]


def _run_norm(st):
    case, x = st["case"], st["x"].float()
    h = x + st["residual"].float() if case["residual"] else x
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * st["weight"].float()
    outs = [y.to(st["x"].dtype)]
    if case["residual"]:
        outs.append(h.to(st["x"].dtype))
    if case["e4m3"]:
        top = y.abs().amax(-1, keepdim=True)
        s = torch.where(top > 0, _over(top, 448.0), 1.0)
        outs += [(y / s).clamp(-448, 448).to(torch.float8_e4m3fn), s[:, 0]]
    return outs


# ----------------------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------------------

def _own_run(st):
    case = st["case"]
    if case["op"] == "norm":
        from segmented_rank_gemm_gb300.norm import rms_norm
        rms_norm(st["x"], st["weight"], 1e-6, residual=st["residual"], residual_out=st["h"],
                 y=st["y"], xq=st["xq"], sx=st["sx"])
        return [st[n] for n in ("y", "h", "xq", "sx") if st[n] is not None]
    if case["op"] == "maps":
        from segmented_rank_gemm_gb300.kv import lora_kv_maps
        lora_kv_maps(st["lens"], st["new"], st["adapter"], case["page"], st["table"], st["free"],
                     st["n_free"], st["kv_len"], st["q_offsets"], st["position"], st["kv_slot"],
                     st["token_slot"], st["counts"])
        return [st[n] for n in ("table", "kv_len", "q_offsets", "position", "kv_slot",
                                "token_slot")] + [st["counts"][:3]]
    if case["op"] == "append":
        st["cache"].append(st["k"], st["v"], st["slots"])
        return list(st["cache"].read(st["slots"], st["k_out"], st["v_out"]))
    return st["cache"].attend(st["q"], st["q_offsets"], st["kv_len"], st["table"], st["max_q"],
                              out=st["out"])


def run(state):
    if own:
        return _own_run(state)
    return {"norm": _run_norm, "maps": _run_maps, "append": _run_append,
            "attend": _run_attend}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------

def _e4m3_64(x):
    """The e4m3 value nearest to each x >= 0 (ties to even), in 64 bits: 4 significant bits
    from 2^-6 up, multiples of 2^-9 below, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(max=448)


def _held_64(x):
    """What the cache holds for bf16 x [T, H, D]."""
    x = x.double().unflatten(-1, (-1, GROUP))
    s = _e4m3_64(x.abs().amax(-1, keepdim=True) / 7)
    n = torch.round(x / torch.where(s > 0, s, 1.0)).clamp(-7, 7)
    return (n * s).flatten(-2)


def exact(case, seed):
    if case["op"] == "maps":
        return None  # whole numbers
    if case["op"] == "norm":
        st = prepare(case, seed)
        h = st["x"].double()
        if case["residual"]:
            h = h + st["residual"].double()
        y = st["weight"].double() * h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / case["k"] + 1e-6)
        outs = [y]
        if case["residual"]:
            outs.append(h)
        if case["e4m3"]:
            s = y.abs().max(-1).values / 448
            s = torch.where(s == 0, 1.0, s)
            outs += [torch.sign(y) * _e4m3_64((y / s[:, None]).abs()), s]
        return outs
    if case["op"] == "append":
        g = _gen(seed)
        t, page = case["tokens"], case["page"]
        k, v = _keys_values(g, t, case["hkv"], case["d"])
        k, v = _held_64(k), _held_64(v)
        if t // 100:
            k[-(t // 100):], v[-(t // 100):] = 0, 0
        return [k, v]
    d = _case_kv(case, seed)
    group, out, k0, q0 = case["hq"] // case["hkv"], [], 0, 0
    for n_kv, n_q in zip(d["kv"], d["new"]):
        k, v = (_held_64(d[x][k0:k0 + n_kv]).permute(1, 0, 2) for x in ("k", "v"))
        q = d["q"][q0:q0 + n_q].double().view(n_q, case["hkv"], group, -1)
        s = torch.einsum("ihgd,hjd->hgij", q, k) / case["d"] ** 0.5
        hidden = torch.ones(n_q, n_kv, dtype=torch.bool, device=DEV).triu(n_kv - n_q + 1)
        p = torch.softmax(s.masked_fill(hidden, float("-inf")), -1)
        out.append(torch.einsum("hgij,hjd->ihgd", p, v).reshape(n_q, case["hq"], case["d"]))
        k0, q0 = k0 + n_kv, q0 + n_q
    return torch.cat(out)
