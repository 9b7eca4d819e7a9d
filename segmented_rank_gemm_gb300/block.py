"""The attention half of a decoder block with an adapter a request, over a 4-bit cache.

    h += x;  n = norm(h) w;  q, k, v = P_q(n), P_k(n), P_v(n);  k, v into the cache
    y = P_o(softmax(scale q K^T) V)

Every projection is a mixed-adapter layer (``lora.LoraLayer``); ``PageTable.step`` gives the
batch's rows their adapter slots, positions and cache slots, so that the requests' lengths and
pages never leave the GPU.  Prompts and single tokens share a batch.  A pass makes no host
synchronisation and, with y given, no allocation, and can be captured in a CUDA graph (with the
batch's ``PageTable.step`` or after it).
"""
from __future__ import annotations

import torch

from .kv import KvCache, PageTable
from .lora import LoraLayer, empty, on_stream
from .norm import lora_rms_norm


class AttentionBlock:
    """``q``, ``k``, ``v`` and ``o`` are LoraLayers: hidden -> q_heads head_dim,
    hidden -> kv_heads head_dim (k and v) and q_heads head_dim -> hidden, in bf16; q, k and v
    all with an e4m3 base, or none of them.  ``norm_weight`` [hidden] is bf16.

    ``rotate(q, k, position)``, if given, turns q [T, q_heads, D] and k [T, kv_heads, D] in
    place before the keys are cached; its torch operations run on the pass's stream."""

    def __init__(self, q: LoraLayer, k: LoraLayer, v: LoraLayer, o: LoraLayer,
                 norm_weight: torch.Tensor, cache: KvCache, eps: float = 1e-6, rotate=None):
        D = cache.head_dim
        if q.N % (cache.kv_heads * D) or q.N > 64 * cache.kv_heads * D \
                or k.N != cache.kv_heads * D or v.N != k.N or o.K != q.N:
            raise ValueError("the projections' widths do not fit the cache's heads")
        if o.N != q.K:
            raise ValueError("o must give rows as wide as the block's")
        if any(layer.dtype != torch.bfloat16 for layer in (q, k, v, o)):
            raise ValueError("the projections must be bf16 layers")
        if not q.K == k.K == v.K or len({layer.fp8_base for layer in (q, k, v)}) != 1:
            raise ValueError("q, k and v must take the same rows")
        self.q, self.k, self.v, self.o = q, k, v, o
        self.norm_weight, self.cache, self.eps, self.rotate = norm_weight, cache, eps, rotate
        self.max_tokens = min(layer.max_tokens for layer in (q, k, v, o))

        def rows(width, dtype=torch.bfloat16):
            return torch.empty(self.max_tokens, width, dtype=dtype, device=norm_weight.device)

        # the batch's intermediate rows; kept, so that a captured graph owns no others
        self.n, self.ctx = rows(q.K), rows(q.N)
        self.qr, self.kr, self.vr = rows(q.N), rows(k.N), rows(v.N)
        self.nq = rows(q.K, torch.float8_e4m3fn) if q.fp8_base else None
        self.sn = rows(1, torch.float32).view(-1) if q.fp8_base else None

    def forward(self, x: torch.Tensor, h: torch.Tensor, pages: PageTable, max_q: int, y=None,
                stream=None) -> torch.Tensor:
        """x and the running residual ``h`` [T, hidden] (overwritten by h + x) of the batch that
        ``pages.step`` mapped last; ``max_q`` bounds a request's new tokens.  Returns y."""
        T = x.shape[0]
        # (whatever can be refused is, before h and the cache change; x and h by the norm)
        if T > min(self.max_tokens, pages.token_slot.shape[0]):
            raise ValueError("more rows than max_tokens")
        if pages.page_size != self.cache.page_size or pages.max_requests > self.cache.max_requests:
            raise ValueError("the page table does not fit the cache")
        if max_q < 1:
            raise ValueError("max_q must be positive")
        if y is None:
            y = empty(x.shape, x.dtype, x.device, stream)
        elif y.dtype != torch.bfloat16 or y.shape != (T, self.o.N) or not y.is_cuda \
                or not y.is_contiguous():
            raise ValueError("y must be a dense CUDA bf16 tensor of x's shape")
        n, nq, sn = self.n[:T], None, None
        if self.nq is not None:
            nq, sn = self.nq[:T], self.sn[:T]
        lora_rms_norm(x, self.norm_weight, self.eps, h, h, n, nq, sn, stream)
        ids = pages.token_slot[:T]
        for layer, rows in ((self.q, self.qr), (self.k, self.kr), (self.v, self.vr)):
            layer.set_batch(ids, stream)
            if nq is None:
                layer.forward(n, rows[:T], stream)
            else:
                layer.forward_e4m3(n, nq, sn, rows[:T], stream)
        D = self.cache.head_dim
        q, k, v, ctx = (r[:T].view(T, r.shape[1] // D, D)
                        for r in (self.qr, self.kr, self.vr, self.ctx))
        if self.rotate is not None:
            with on_stream(stream):
                self.rotate(q, k, pages.position[:T])
        self.cache.append(k, v, pages.kv_slot[:T], stream)
        self.cache.attend(q, pages.q_offsets, pages.kv_len, pages.block_table, max_q, out=ctx,
                          stream=stream)
        self.o.set_batch(ids, stream)
        return self.o.forward(self.ctx[:T], y, stream)
