"""More operators of a multi-adapter decoder block, as cases to measure.

- ``rotate``  new tokens' queries and keys turned by their positions, keys and values written
              to the 4-bit paged cache on the way (and read back)
- ``shared``  causal attention of a batch whose requests share long prefixes by groups
- ``cross``   attention of a decoder's tokens to all of their request's encoder states
- ``fused``   a mixed-adapter product with bias, activation, a factor and a residual:
              y = act(x W + s (x A) B + bias) * factor + residual

``run`` computes them in plain torch operations in 32 bits; with ``own`` set it makes the calls of
``segmented_rank_gemm_gb300.kv`` and ``segmented_rank_gemm_gb300.lora``.

The 4-bit format: 16 consecutive dimensions of one token and head share one scale
s = e4m3(max|x| / 7); codes are round(x / s) in -7..7, kept with 8 added, and stand for code * s.
Keys are rotated in 32 bits and quantised from there.
"""
import math
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
        # a single user's next token, far into a document: the smallest call
        {"name": "rotate_one", "op": "rotate", "tokens": 1, "positions": 131072, "rotary": 128,
         "interleaved": False, **HEADS},
        # the stack's decode batch: one token a request, positions all over the table
        {"name": "rotate_512", "op": "rotate", "tokens": 512, "positions": 8192, "rotary": 128,
         "interleaved": False, **HEADS},
        # the prefill workload's token count, with padding rows
        {"name": "rotate_8192", "op": "rotate", "tokens": 8192, "positions": 32768, "rotary": 128,
         "interleaved": False, **HEADS},
        # four samples of one question: the fewest rows that share
        {"name": "shared_four", "op": "shared", "requests": 4, "groups": 1, "prefix": 1024,
         "tail": 64, "chunk": 1, **HEADS},
        # the stack's decode batch, a system prompt for each of eight adapters
        {"name": "shared_decode_512", "op": "shared", "requests": 512, "groups": 8, "prefix": 2048,
         "tail": 512, "chunk": 1, **HEADS},
        # many questions on one long document
        {"name": "shared_document", "op": "shared", "requests": 64, "groups": 1, "prefix": 32768,
         "tail": 1024, "chunk": 1, **HEADS},
        # drafts of several tokens to verify, small pages, groups of uneven size
        {"name": "shared_drafts", "op": "shared", "requests": 61, "groups": 5, "prefix": 4096,
         "tail": 300, "chunk": 7, "hq": 32, "hkv": 8, "d": 128, "page": 16},
        # a decode step of an encoder-decoder model, ragged encoder lengths
        {"name": "cross_decode_256", "op": "cross", "requests": 256, "chunk": 1, "ctx": 1500,
         **HEADS},
        # its decoder prompts
        {"name": "cross_prompts", "op": "cross", "requests": 16, "chunk": 448, "ctx": 1500,
         **HEADS},
        # the stack's down projection at decode: bias and the running residual
        {"name": "fused_down_512", "op": "fused", "tokens": 512, "k": 14336, "n": 4096,
         "slots": 100, "rank": 16, "act": "none", "bias": True, "factor": False, "residual": True,
         "e4m3": False},
        # its gate projection from an e4m3 base: SiLU and the product with the up projection
        {"name": "fused_gate_512_e4m3", "op": "fused", "tokens": 512, "k": 4096, "n": 14336,
         "slots": 100, "rank": 16, "act": "silu", "bias": False, "factor": True, "residual": False,
         "e4m3": True},
        # the prefill workload's gate projection
        {"name": "fused_gate_8192", "op": "fused", "tokens": 8192, "k": 4096, "n": 14336,
         "slots": 32, "rank": 16, "act": "silu", "bias": False, "factor": True, "residual": False,
         "e4m3": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("rotate", "shared", "shared", "cross", "fused", "fused"))
    if op == "fused":
        k, n = 16 * _log_int(rng, 8, 896), 8 * _log_int(rng, 16, 1792)
        # (the largest listed product bounds the rows)
        rows = min(8192, 8192 * 4096 * 14336 // (k * n))
        return {"op": op, "tokens": _log_int(rng, 1, rows), "k": k, "n": n,
                "slots": _log_int(rng, 1, 32), "rank": rng.choice((4, 8, 16, 24, 64)),
                "act": rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")),
                "bias": rng.random() < 0.5, "factor": rng.random() < 0.5,
                "residual": rng.random() < 0.5, "e4m3": rng.random() < 0.4}
    heads = {"hkv": rng.choice((1, 2, 3, 4, 8)), "d": rng.choice((64, 128)),
             "page": rng.choice((16, 32, 64, 128))}
    heads["hq"] = heads["hkv"] * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * heads["hkv"] <= 32])
    if op == "rotate":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "positions": _log_int(rng, 64, 131072),
                "rotary": rng.choice((heads["d"], heads["d"], heads["d"] // 2, 32)),
                "interleaved": rng.random() < 0.4, **heads}
    if op == "cross":
        chunk = rng.choice((1, 1, _log_int(rng, 2, 448)))
        most = 256 if chunk == 1 else max(1, min(256, 16 * 448 // chunk))
        return {"op": op, "requests": _log_int(rng, 1, most), "chunk": chunk,
                "ctx": _log_int(rng, 16, 1500), **heads}
    kind = rng.choice(("decodes", "decodes", "document", "drafts"))
    if kind == "document":
        n = _log_int(rng, 2, 64)
        return {"op": op, "requests": n, "groups": rng.randint(1, min(3, n)),
                "prefix": _log_int(rng, 2048, 32768), "tail": _log_int(rng, 1, 1024), "chunk": 1,
                **heads}
    n = _log_int(rng, 2, 512 if kind == "decodes" else 61)
    return {"op": op, "requests": n, "groups": _log_int(rng, 1, min(n, 40)),
            "prefix": _log_int(rng, 128, 2048), "tail": _log_int(rng, 1, 512),
            "chunk": 1 if kind == "decodes" else rng.randint(2, 7), **heads}


# ----------------------------------------------------------------------------------------
# lengths: a function of the case alone, so that work() is exact
# ----------------------------------------------------------------------------------------

def _cdiv(a, b):
    return -(-a // b)


def _lengths(case):
    """Of a shared or cross case: (first request of each group and the end, the group's shared
    positions, each request's cached positions with the new ones, its new tokens)."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["requests"]
    new = [rng.randint(_cdiv(case["chunk"], 2), case["chunk"]) for _ in range(n)]
    new[0] = case["chunk"]
    if case["op"] == "cross":
        # an empty encoder now and then; the first is the longest
        kv = [0 if rng.random() < 0.02 else rng.randint(_cdiv(case["ctx"], 8), case["ctx"])
              for _ in range(n)]
        kv[0] = case["ctx"]
        return [0, n], [0], kv, new
    first = [0] + sorted(rng.sample(range(1, n), case["groups"] - 1)) + [n]
    page, shared, kv = case["page"], [], []
    for g in range(case["groups"]):
        blocks = case["prefix"] // page
        if g:  # some groups share less, some nothing
            blocks = 0 if rng.random() < 0.1 else rng.randint(_cdiv(blocks, 2), blocks)
        shared.append(blocks * page)
        for b in range(first[g], first[g + 1]):
            tail = _log_int(rng, 1, case["tail"]) if b else case["tail"]
            kv.append(shared[g] + tail - 1 + new[b])
    return first, shared, kv, new


def work(case):
    if case["op"] == "fused":
        t, k, n, size = case["tokens"], case["k"], case["n"], 1 if case["e4m3"] else 2
        used = min(t, case["slots"])
        rows = 1 + case["factor"] + case["residual"]  # y in and out
        return {"bytes": 2 * t * k + size * k * n + 2 * used * case["rank"] * (k + n) + 2 * rows * t * n
                + (2 * n if case["bias"] else 0) + 4 * t,
                "flops": 2 * t * k * n + 2 * t * case["rank"] * (k + n)}
    if case["op"] == "rotate":
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        q, n = t * hq * d, 2 * t * hkv * d
        # q in and out; k and v in, codes and scales written, values read back from them; angles
        return {"bytes": 4 * q + n * 2 + n // 2 + n // GROUP + n * 2 + 8 * t
                + min(t, case["positions"]) * case["rotary"] * 4,
                "flops": 3 * (q + n // 2) * case["rotary"] // d + 4 * n}
    first, shared, kv, new = _lengths(case)
    held = pairs = 0
    for g, s in enumerate(shared):
        held += s if first[g + 1] > first[g] else 0
        for b in range(first[g], first[g + 1]):
            held += kv[b] - s
            pairs += new[b] * kv[b] - (new[b] * (new[b] - 1) // 2 if case["op"] == "shared" else 0)
    cache = held * case["hkv"] * case["d"] * 2 * (0.5 + 1 / GROUP)
    return {"bytes": int(cache) + 2 * 2 * sum(new) * case["hq"] * case["d"],
            "flops": 4 * pairs * case["hq"] * case["d"]}


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _keys_values(g, tokens, hkv, d):
    """Keys with channels of very different size, as projections give them, and plain values."""
    size = torch.exp(0.7 * _randn(g, hkv, d))
    k = (_randn(g, tokens, hkv, d) * size).bfloat16()
    v = (_randn(g, tokens, hkv, d) * 0.5).bfloat16()
    return k, v


def _case_kv(case, seed):
    """Of a shared or cross case: queries, the block table over shuffled pages, and the cached
    tokens (the groups' prefixes, then the requests' own) with their cache slots."""
    g = _gen(seed)
    first, shared, kv, new = _lengths(case)
    page, n = case["page"], case["requests"]
    group = np.repeat(np.arange(len(shared)), np.diff(first))
    share = np.asarray(shared)[group]
    runs = list(shared) + [a - int(s) for a, s in zip(kv, share)]  # positions of each run of pages
    blocks = np.asarray([_cdiv(r, page) for r in runs])
    start = np.concatenate(([0], np.cumsum(blocks)))
    pages = int(start[-1]) + 3
    order = torch.randperm(pages, generator=g, device=DEV).int()
    col = np.arange(max(1, max(_cdiv(a, page) for a in kv)))[None, :]
    n_pre = (share // page)[:, None]
    own_run = len(shared) + np.arange(n)
    at = np.where(col < n_pre, start[group][:, None] + col, start[own_run][:, None] + col - n_pre)
    at = np.where(col < n_pre + blocks[own_run][:, None], at, pages - 1)
    table = order[torch.from_numpy(at).to(DEV)].contiguous()
    # slots of the runs' tokens, in order
    count = np.asarray(runs)
    run = np.repeat(np.arange(len(runs)), count)
    pos = np.arange(count.sum()) - np.repeat(np.cumsum(count) - count, count)
    block = torch.from_numpy(start[run] + pos // page).to(DEV)
    slots = (order[block].long() * page + torch.from_numpy(pos % page).to(DEV)).int()
    k, v = _keys_values(g, len(run), case["hkv"], case["d"])
    q = _randn(g, sum(new), case["hq"], case["d"]).bfloat16()
    return {"q": q, "table": table, "pages": pages, "k": k, "v": v, "slots": slots, "kv": kv,
            "new": new, "first": first, "shared": shared, "share": share, "runs": runs,
            "group": group}


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


def _fused_inputs(case, seed):
    g = _gen(seed)
    t, k, n, r, s = (case[x] for x in ("tokens", "k", "n", "rank", "slots"))
    d = {"x": _randn(g, t, k).bfloat16(), "W": (_randn(g, k, n) * k ** -0.5).bfloat16(),
         "A": (_randn(g, s, k, r) * k ** -0.5).bfloat16(),
         "B": (_randn(g, s, r, n) * r ** -0.5).bfloat16(), "alpha": 2.0 * r}
    ids = torch.randint(0, s, (t,), generator=g, device=DEV).int()
    if t > 512:  # prompts: runs of tokens of one adapter
        ids = ids.sort().values
    d["ids"] = torch.where(torch.rand(t, generator=g, device=DEV) < 0.1, -1, ids).int()
    d["bias"] = _randn(g, n).bfloat16() if case["bias"] else None
    d["factor"] = _randn(g, t, n).bfloat16() if case["factor"] else None
    d["residual"] = (_randn(g, t, n) * 4).bfloat16() if case["residual"] else None
    return d


def _rotate_inputs(case, seed):
    g = _gen(seed)
    t, page = case["tokens"], case["page"]
    pages = _cdiv(t, page) * 2 + 1
    k, v = _keys_values(g, t, case["hkv"], case["d"])
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:t].int()
    slots[t - t // 100:] = -1  # padding rows
    # (far positions, whatever the table's length)
    position = torch.randint(0, case["positions"], (t,), generator=g, device=DEV).int()
    position[0] = case["positions"] - 1
    return {"q": _randn(g, t, case["hq"], case["d"]).bfloat16(), "k": k, "v": v, "slots": slots,
            "position": position, "pages": pages}


def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "fused":
        st.update(_fused_inputs(case, seed))
        st["y"] = torch.empty(case["tokens"], case["n"], dtype=torch.bfloat16, device=DEV)
        W, A, B = st.pop("W"), st.pop("A"), st.pop("B")
        if own:
            from segmented_rank_gemm_gb300.lora import LoraLayer
            st["layer"] = LoraLayer(W, case["slots"], case["rank"], case["tokens"],
                                    fp8_base=case["e4m3"])
            for i in range(case["slots"]):
                st["layer"].load(i, A[i], B[i], st["alpha"])
        else:
            # adapters side by side: slot s has columns (rows) s r .. s r + r - 1
            st["A"], st["B"] = A.transpose(0, 1).flatten(1).contiguous(), B.flatten(0, 1)
            st["W"] = W
            if case["e4m3"]:
                w = W.float()
                top = w.abs().amax(0, keepdim=True)
                st["sw"] = torch.where(top > 0, _over(top, 448.0), 1.0)
                st["W"] = (w / st["sw"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return st
    if case["op"] == "rotate":
        st.update(_rotate_inputs(case, seed))
        st["q_out"] = torch.empty_like(st["q"])
        st["k_out"], st["v_out"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        if own:
            from segmented_rank_gemm_gb300.kv import Rotary
            st["rotary"] = Rotary(case["positions"], case["rotary"], theta=10000.0,
                                  interleaved=case["interleaved"])
            st["cache"] = _own_cache(st["pages"], case, 1)
        else:
            angle = _angles(torch.arange(case["positions"], device=DEV), case["rotary"])
            st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
            st["pool"] = _pool(st["pages"], case)
        return st
    d = _case_kv(case, seed)
    st.update(q=d["q"], table=d["table"], kv_len=_ints(d["kv"]), max_q=max(d["new"]),
              q_offsets=_ints(np.concatenate(([0], np.cumsum(d["new"]))).tolist()),
              max_kv=max(d["kv"]), group_offsets=_ints(d["first"]),
              prefix_row=_ints(d["first"][:-1]), prefix_len=_ints(d["shared"]),
              shared=_ints(d["share"].tolist()), out=torch.empty_like(d["q"]))
    if own:
        st["cache"] = _own_cache(d["pages"], case, case["requests"])
        st["cache"].append(d["k"], d["v"], d["slots"])
        if case["op"] == "shared":
            st["workspace"] = st["cache"].shared_workspace(d["q"].shape[0], case["hq"])
    else:
        st["pool"] = _pool(d["pages"], case)
        _append(st["pool"], d["k"].float(), d["v"].float(), d["slots"])
    return st


# ----------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------

def _over(x, n):
    """x / n, correctly rounded (a division by a Python number multiplies by its reciprocal,
    which turns quotients halfway between two e4m3 values to one side)."""
    return x / torch.full_like(x, n)


def _angles(position, rotary):
    """Angles [.., rotary / 2] in 64 bits: position * 10000^(-2 i / rotary)."""
    i = torch.arange(rotary // 2, device=DEV, dtype=torch.float64)
    return position.double()[..., None] * torch.exp(i * (-2 * math.log(10000.0) / rotary))


def _quantize(x):
    """fp32 [T, H, D] -> packed codes [T, H, D/2] and e4m3 scales [T, H, D/16]."""
    x = x.unflatten(-1, (-1, GROUP))
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


def _turn(x, cos, sin, rotary, interleaved):
    """The first `rotary` dimensions of x [T, H, D] turned by [T, rotary / 2] angles: pairs
    (i, i + rotary / 2), or (2 i, 2 i + 1)."""
    x, cos, sin = x.float(), cos[:, None, :], sin[:, None, :]
    head = x[..., :rotary]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :rotary // 2], head[..., rotary // 2:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((head, x[..., rotary:]), -1)


def _run_rotate(st):
    case, pool, slots = st["case"], st["pool"], st["slots"]
    p = st["position"].long()
    cos, sin = st["cos"][p], st["sin"][p]
    q = _turn(st["q"], cos, sin, case["rotary"], case["interleaved"])
    k = _turn(st["k"], cos, sin, case["rotary"], case["interleaved"])
    _append(pool, k, st["v"].float(), slots)
    at, there = slots.clamp(min=0).long(), (slots >= 0)[:, None, None]
    held = [torch.where(there, _rows(pool[c], pool[s], at), 0.0).bfloat16()
            for c, s in (("kc", "ks"), ("vc", "vs"))]
    return [q.bfloat16()] + held


def _run_attend(st):
    """Every request over all that it sees, padded to the longest."""
    case, pool = st["case"], st["pool"]
    page, hkv, d, max_q = case["page"], case["hkv"], case["d"], st["max_q"]
    group, n, t = case["hq"] // hkv, case["requests"], st["q"].shape[0]
    kv_len, first = st["kv_len"].long(), st["q_offsets"][:-1].long()
    q_len = st["q_offsets"][1:].long() - first
    pos = torch.arange(st["max_kv"], device=DEV)
    slot = st["table"].long()[:, pos // page] * page + pos % page
    k = _rows(pool["kc"], pool["ks"], slot).permute(0, 2, 3, 1)  # [n, hkv, d, L]
    i = torch.arange(max_q, device=DEV)
    q = st["q"][(first[:, None] + i).clamp(max=t - 1)].float()  # [n, max_q, hq, d]
    q = q.view(n, max_q, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * max_q, d)
    s = torch.matmul(q, k) * d ** -0.5
    last = (kv_len - 1)[:, None].expand(n, max_q)  # the last position a query sees
    if case["op"] == "shared":
        last = last + 1 - q_len[:, None] + i
    seen = pos <= last[:, :, None]  # [n, max_q, L]
    s = s.view(n, hkv, group, max_q, -1).masked_fill(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1)
    v = _rows(pool["vc"], pool["vs"], slot).permute(0, 2, 1, 3)  # [n, hkv, L, d]
    o = torch.matmul(p.view(n, hkv, group * max_q, -1), v).view(n, hkv, group, max_q, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, max_q, case["hq"], d)
    token = torch.arange(t, device=DEV)
    b = torch.searchsorted(first + q_len, token, right=True)
    return o[b, token - first[b]].bfloat16()


def _act(x, name):
    if name == "relu":
        return x.clamp(min=0)
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x ** 3)))
    return x


def _run_fused(st):
    case, x, ids = st["case"], st["x"].float(), st["ids"]
    if case["e4m3"]:
        top = x.abs().amax(-1, keepdim=True)
        sx = torch.where(top > 0, _over(top, 448.0), 1.0)
        xq = (x / sx).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        y = (xq @ st["W"].float()) * sx * st["sw"]
    else:
        y = x @ st["W"].float()
    slot = torch.arange(case["slots"], device=DEV).repeat_interleave(case["rank"])
    v = (x @ st["A"].float()) * (st["alpha"] / case["rank"])
    y = y + torch.where(slot == ids[:, None], v, 0.0) @ st["B"].float()
    if case["bias"]:
        y = y + st["bias"].float()
    y = _act(y, case["act"])
    if case["factor"]:
        y = y * st["factor"].float()
    if case["residual"]:
        y = y + st["residual"].float()
    return y.bfloat16()


# ----------------------------------------------------------------------------------------
# the framework's calls
# ----------------------------------------------------------------------------------------

def _own_run(st):
    case = st["case"]
    if case["op"] == "fused":
        st["layer"].set_batch(st["ids"])
        return st["layer"].forward_fused(st["x"], st["y"], bias=st["bias"], activation=case["act"],
                                         factor=st["factor"], residual=st["residual"])
    cache = st["cache"]
    if case["op"] == "rotate":
        cache.append_rotated(st["q"], st["k"], st["v"], st["position"], st["slots"], st["rotary"],
                             q_out=st["q_out"])
        return [st["q_out"], *cache.read(st["slots"], st["k_out"], st["v_out"])]
    if case["op"] == "cross":
        return cache.attend(st["q"], st["q_offsets"], st["kv_len"], st["table"], st["max_q"],
                            out=st["out"], causal=False)
    return cache.attend_shared(st["q"], st["q_offsets"], st["kv_len"], st["table"], st["max_q"],
                               st["group_offsets"], st["prefix_row"], st["prefix_len"],
                               st["shared"], out=st["out"], workspace=st["workspace"])


def run(state):
    if own:
        return _own_run(state)
    return {"rotate": _run_rotate, "shared": _run_attend, "cross": _run_attend,
            "fused": _run_fused}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------

def _e4m3_64(x):
    """The e4m3 value nearest to each x >= 0 (ties to even), in 64 bits: 4 significant bits
    from 2^-6 up, multiples of 2^-9 below, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(max=448)


def _held_64(x):
    """What the cache holds for x [T, H, D] in 64 bits."""
    x = x.unflatten(-1, (-1, GROUP))
    s = _e4m3_64(x.abs().amax(-1, keepdim=True) / 7)
    n = torch.round(x / torch.where(s > 0, s, 1.0)).clamp(-7, 7)
    return (n * s).flatten(-2)


def _exact_rotate(case, seed):
    d = _rotate_inputs(case, seed)
    angle = _angles(d["position"], case["rotary"])

    def turned(x):  # as a product of complex numbers
        z, r = x.double(), case["rotary"]
        pairs = (z[..., :r].unflatten(-1, (-1, 2)) if case["interleaved"]
                 else z[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)).contiguous()
        w = torch.view_as_real(torch.view_as_complex(pairs)
                               * torch.polar(torch.ones_like(angle), angle)[:, None])
        w = (w if case["interleaved"] else w.transpose(-1, -2)).flatten(-2)
        return torch.cat((w, z[..., r:]), -1)

    there = (d["slots"] >= 0).double()[:, None, None]
    return [turned(d["q"]), _held_64(turned(d["k"])) * there, _held_64(d["v"].double()) * there]


def _exact_fused(case, seed):
    d = _fused_inputs(case, seed)
    x, W = d["x"].double(), d["W"].double()
    if case["e4m3"]:
        sx, sw = (w.abs().amax(i, keepdim=True) / 448 for w, i in ((x, 1), (W, 0)))
        sx, sw = torch.where(sx > 0, sx, 1.0), torch.where(sw > 0, sw, 1.0)
        xq, wq = x / sx, W / sw
        y = ((torch.sign(xq) * _e4m3_64(xq.abs())) @ (torch.sign(wq) * _e4m3_64(wq.abs()))) * sx * sw
    else:
        y = x @ W
    for s in d["ids"].unique().tolist():
        if s >= 0:
            rows = (d["ids"] == s).nonzero()[:, 0]
            y[rows] += 2.0 * (x[rows] @ d["A"][s].double()) @ d["B"][s].double()  # alpha / rank
    if case["bias"]:
        y += d["bias"].double()
    y = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[case["act"]](y)
    if case["factor"]:
        y *= d["factor"].double()
    if case["residual"]:
        y += d["residual"].double()
    return y


def exact(case, seed):
    if case["op"] == "rotate":
        return _exact_rotate(case, seed)
    if case["op"] == "fused":
        return _exact_fused(case, seed)
    d = _case_kv(case, seed)
    k, v = _held_64(d["k"].double()), _held_64(d["v"].double())
    at = np.concatenate(([0], np.cumsum(d["runs"]))).tolist()
    groups, q0, out = len(d["shared"]), 0, []
    for b, (n_kv, n_q) in enumerate(zip(d["kv"], d["new"])):
        g, run_b = int(d["group"][b]), groups + b
        kb, vb = (torch.cat((x[at[g]:at[g + 1]], x[at[run_b]:at[run_b + 1]])).transpose(0, 1)
                  for x in (k, v))
        q = d["q"][q0:q0 + n_q].double().view(n_q, case["hkv"], -1, case["d"])
        s = torch.einsum("ihgd,hjd->hgij", q, kb) / case["d"] ** 0.5
        if case["op"] == "shared":
            hidden = torch.ones(n_q, n_kv, dtype=torch.bool, device=DEV).triu(n_kv - n_q + 1)
            s = s.masked_fill(hidden, float("-inf"))
        o = torch.einsum("hgij,hjd->ihgd", torch.softmax(s, -1), vb)
        out.append(o.reshape(n_q, case["hq"], case["d"]))
        q0 += n_q
    return torch.cat(out)
