"""Plain definitions, in numpy and 64 bits, of the steps between a block's projections: the
4-bit cache's values, attention over them, block tables and slot maps, and the residual norm.
Test infrastructure: written from the definitions, without the library's code."""
from __future__ import annotations

import numpy as np

GROUP = 16

# the 127 finite non-negative e4m3 values, ascending: value of code c
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                 for c in range(127)])


def to_e4m3(x):
    """Nearest e4m3 value of each x >= 0, ties to the even code, at most 448 (64-bit input)."""
    x = np.minimum(np.asarray(x, np.float64), E4M3[-1])
    hi = np.clip(np.searchsorted(E4M3, x), 1, len(E4M3) - 1)
    lo = hi - 1
    dl, dh = x - E4M3[lo], E4M3[hi] - x
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return E4M3[pick]


def held(x, g=1.0):
    """The values a cache of scale g holds for x [..., D] (any float type, bf16 values): scale
    and quotient are fp32 divisions, correctly rounded."""
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), x)
    g = np.float32(g)
    grp = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    with np.errstate(all="ignore"):
        s8 = to_e4m3((np.abs(grp).max(-1) / (np.float32(7) * g)).astype(np.float32))
        s = s8.astype(np.float32) * g
        n = np.rint(grp / np.where(s > 0, s, np.float32(1))[..., None])
    n = np.where((s > 0)[..., None], np.clip(n, -7, 7), 0)
    # the value: the fp32 product n s8 g, n s8 being exact
    v = (n * s8[..., None]).astype(np.float32) * g
    return v.reshape(x.shape).astype(np.float64)


def attend(q, k, v, scale):
    """q [n, Hq, D] the last n positions' queries; k, v [L, Hkv, D]: [n, Hq, D] in 64 bits.
    Query i sees positions 0 .. L - n + i; one that sees nothing gives zeros."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, hq, d = q.shape
    L, hkv = k.shape[:2]
    out = np.zeros((n, hq, d))
    for h in range(hq):
        kv = h // (hq // hkv)
        if L == 0:
            continue
        s = scale * q[:, h] @ k[:, kv].T
        seen = np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]
        for i in range(n):
            if seen[i].any():
                w = np.exp(s[i, seen[i]] - s[i, seen[i]].max())
                out[i, h] = (w / w.sum()) @ v[seen[i], kv]
    return out


def attend_all(q, k, v, scale):
    """As ``attend`` without the causal mask: every query sees all L positions (none: zeros)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out = np.zeros(q.shape)
    group = q.shape[1] // k.shape[1]
    for h in range(q.shape[1] if len(k) else 0):
        s = scale * q[:, h] @ k[:, h // group].T
        w = np.exp(s - s.max(-1, keepdims=True))
        out[:, h] = (w / w.sum(-1, keepdims=True)) @ v[:, h // group]
    return out


def rotated(x, cos, sin, interleaved, dtype=np.float32):
    """x [T, H, D] with its first dimensions turned by angles of [T, R / 2] cosines and sines, pairs
    (i, i + R / 2) or (2 i, 2 i + 1): (a c - b s, b c + a s), each operation in ``dtype``."""
    x = np.asarray(x, dtype)
    cos, sin = (np.asarray(c, dtype)[:, None, :] for c in (cos, sin))
    half = cos.shape[-1]
    at = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if interleaved else (
        np.arange(half), np.arange(half, 2 * half))
    out = x.copy()
    with np.errstate(all="ignore"):
        a, b = x[..., at[0]], x[..., at[1]]
        out[..., at[0]] = a * cos - b * sin
        out[..., at[1]] = b * cos + a * sin
    return out


def maps(lens, new, adapter, page, table, free, n_free, T):
    """lora_kv_maps in plain Python.  Returns the dict of its outputs (table a copy)."""
    B, blocks = table.shape
    num_pages = (2 ** 31 - 1) // page  # ids whose slots are 32-bit
    table = table.copy()
    cdiv = lambda a: -(-a // page)  # noqa: E731
    flags = 0
    if any(a < 0 or b < 0 or a + b > blocks * page for a, b in zip(lens, new)):
        flags |= 1
    good = [(a, b) if a >= 0 and b >= 0 and a + b <= blocks * page else (0, 0)
            for a, b in zip(lens, new)]
    if sum(b for _, b in good) > T:
        flags |= 1
    need = sum(cdiv(a + b) - cdiv(a) for a, b in good)
    if n_free < 0 or n_free > len(free) or need > n_free:
        flags |= 2
    out = {"table": table, "kv_len": list(lens), "q_offsets": [0] * (B + 1), "position": [0] * T,
           "kv_slot": [-1] * T, "token_slot": [-1] * T, "counts": [0, n_free, 0, flags, 0]}
    if flags:
        return out
    top, row = n_free, 0
    for b in range(B):
        for blk in range(cdiv(lens[b]), cdiv(lens[b] + new[b])):
            top -= 1
            table[b, blk] = free[top]
        for i in range(new[b]):
            pos = lens[b] + i
            p = int(table[b, pos // page])
            out["position"][row] = pos
            out["token_slot"][row] = -1 if adapter is None else int(adapter[b])
            if 0 <= p < num_pages:
                out["kv_slot"][row] = p * page + pos % page
            else:
                flags |= 4
            row += 1
        out["kv_len"][b] = lens[b] + new[b]
        out["q_offsets"][b + 1] = row
        for blk in range(cdiv(lens[b]), cdiv(lens[b] + new[b])):
            if not 0 <= table[b, blk] < num_pages:
                flags |= 4
    out["counts"] = [row, top, n_free - top, flags, 0]
    return out


def rms_norm(x, residual, w, eps):
    """(h, y, sx) in 64 bits."""
    h = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    top = np.abs(y).max(-1)
    return h, y, np.where(top > 0, top / 448, 1.0)
