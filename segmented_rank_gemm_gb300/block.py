"""The two halves of a decoder block with an adapter a request, the first over a 4-bit cache.

    h += x;  n = norm(h) w;  q, k, v = P_q(n), P_k(n), P_v(n);  k, v into the cache
    y = P_o(softmax(scale q K^T) V)

    h += y;  n = norm(h) w;  z = P_down(act(P_gate(n)) * P_up(n))

Every projection is a mixed-adapter layer (``lora.LoraLayer``); ``PageTable.step`` gives the
batch's rows their adapter slots, positions and cache slots, so that the requests' lengths and
pages never leave the GPU.  Prompts and single tokens share a batch.  A pass makes no host
synchronisation and, with y given, no allocation, and can be captured in a CUDA graph (with the
batch's ``PageTable.step`` or after it).
"""
from __future__ import annotations

import torch

from .kv import KvCache, PageTable, Rotary
from .lora import ACTIVATIONS, LoraLayer, empty, on_stream
from .norm import lora_rms_norm


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether the memory from the first to the last element of two arrays of rows meets."""
    if not a.numel() or not b.numel():
        return False
    (a0, a1), (b0, b1) = ((t.data_ptr(), t.data_ptr() + t.element_size() * (
        1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))) for t in (a, b))
    return a0 < b1 and b0 < a1


def _product(layer: LoraLayer, x, y, xq, sx, stream) -> torch.Tensor:
    """A product with nothing in its epilogue.  Rows of an e4m3 base leave by whole lines in a fused
    forward's epilogue, which pays beyond decode batches (8192 rows 4096 -> 14336 419 us, 431 by the plain
    forward; 512 rows 75 and 72).  A bf16 base's take 2% less by the plain one, the same at 512 rows."""
    if layer.fp8_base and x.shape[0] > 512:
        return layer.forward_fused(x, y, xq=xq, sx=sx, stream=stream)
    if xq is None:
        return layer.forward(x, y, stream)
    return layer.forward_e4m3(x, xq, sx, y, stream)


class AttentionBlock:
    """``q``, ``k``, ``v`` and ``o`` are LoraLayers: hidden -> q_heads head_dim,
    hidden -> kv_heads head_dim (k and v) and q_heads head_dim -> hidden, in bf16; q, k and v
    all with an e4m3 base, or none of them.  ``norm_weight`` [hidden] is bf16.

    ``rotary``, if given, turns queries and keys by their positions on the way into the cache.
    ``rotate(q, k, position)``, if given instead, turns q [T, q_heads, D] and k [T, kv_heads, D] in
    place before the keys are cached; its torch operations run on the pass's stream.  ``share``:
    passes may be given groups of requests that share prefixes."""

    def __init__(self, q: LoraLayer, k: LoraLayer, v: LoraLayer, o: LoraLayer,
                 norm_weight: torch.Tensor, cache: KvCache, eps: float = 1e-6, rotate=None,
                 rotary: Rotary = None, share: bool = False):
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
        if rotary is not None and (rotate is not None or rotary.rotary_dim > D
                                   or rotary.angles.device != norm_weight.device):
            raise ValueError("rotate or a rotary of at most the head's dimensions, on the block's device")
        self.q, self.k, self.v, self.o = q, k, v, o
        self.norm_weight, self.cache, self.eps, self.rotate = norm_weight, cache, eps, rotate
        self.rotary = rotary
        self.max_tokens = min(layer.max_tokens for layer in (q, k, v, o))

        def rows(width, dtype=torch.bfloat16):
            return torch.empty(self.max_tokens, width, dtype=dtype, device=norm_weight.device)

        # the batch's intermediate rows; kept, so that a captured graph owns no others
        self.n, self.ctx = rows(q.K), rows(q.N)
        self.qr, self.kr, self.vr = rows(q.N), rows(k.N), rows(v.N)
        self.nq = rows(q.K, torch.float8_e4m3fn) if q.fp8_base else None
        self.sn = rows(1, torch.float32).view(-1) if q.fp8_base else None
        self.parts = cache.shared_workspace(self.max_tokens, q.N // D) if share else None

    def forward(self, x: torch.Tensor, h: torch.Tensor, pages: PageTable, max_q: int, y=None,
                stream=None, groups=None) -> torch.Tensor:
        """x and the running residual ``h`` [T, hidden] (overwritten by h + x) of the batch that
        ``pages.step`` mapped last; ``max_q`` bounds a request's new tokens.  Returns y, which does not
        overlap h.
        ``groups``: (group_offsets, prefix_row, prefix_len) of ``KvCache.attend_shared``, whose
        members' prefixes are ``pages.shared_len``."""
        T = x.shape[0]
        # (whatever can be refused is, before h and the cache change; x and h by the norm)
        if T > min(self.max_tokens, pages.token_slot.shape[0]):
            raise ValueError("more rows than max_tokens")
        if pages.page_size != self.cache.page_size or pages.max_requests > self.cache.max_requests:
            raise ValueError("the page table does not fit the cache")
        if max_q < 1:
            raise ValueError("max_q must be positive")
        if groups is not None:
            if self.parts is None:
                raise ValueError("groups need a block made with share")
            self.cache.check_groups(pages.max_requests, *groups)
        if y is None:
            y = empty(x.shape, x.dtype, x.device, stream)
        elif y.dtype != torch.bfloat16 or y.shape != (T, self.o.N) or y.device != x.device \
                or not y.is_contiguous() or y.data_ptr() % 16:
            raise ValueError("y must be a dense, 16-byte aligned bf16 tensor of x's shape on x's device")
        elif _overlap(y, h):
            raise ValueError("y and h overlap")
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
        if self.rotary is not None:
            self.cache.append_rotated(q, k, v, pages.position[:T], pages.kv_slot[:T], self.rotary,
                                      q_out=q, stream=stream)
        else:
            if self.rotate is not None:
                with on_stream(stream):
                    self.rotate(q, k, pages.position[:T])
            self.cache.append(k, v, pages.kv_slot[:T], stream)
        batch = (q, pages.q_offsets, pages.kv_len, pages.block_table, max_q)
        if groups is None:
            self.cache.attend(*batch, out=ctx, stream=stream)
        else:
            self.cache.attend_shared(*batch, *groups, pages.shared_len, out=ctx,
                                     workspace=self.parts, stream=stream)
        self.o.set_batch(ids, stream)
        return self.o.forward(self.ctx[:T], y, stream)


class MlpBlock:
    """``gate``, ``up`` and ``down`` are LoraLayers: hidden -> width (gate and up) and width ->
    hidden, in bf16; gate and up both with an e4m3 base, or neither.  ``norm_weight`` [hidden] is
    bf16; ``activation`` one of ``lora.ACTIVATIONS``.

    The gate's product ends in act(.) times the up projection's rows, and, in a pass with
    ``residual``, the down projection's in the sum with h: three products and a norm, no other
    pass over the rows."""

    def __init__(self, gate: LoraLayer, up: LoraLayer, down: LoraLayer, norm_weight: torch.Tensor,
                 activation: str = "silu", eps: float = 1e-6):
        if not (gate.K == up.K == down.N and gate.N == up.N == down.K):
            raise ValueError("gate and up must give the rows that down takes, down rows like theirs")
        if any(layer.dtype != torch.bfloat16 for layer in (gate, up, down)):
            raise ValueError("the projections must be bf16 layers")
        if gate.fp8_base != up.fp8_base:
            raise ValueError("gate and up must take the same rows")
        if activation not in ACTIVATIONS:
            raise ValueError("activation must be one of %s" % sorted(filter(None, ACTIVATIONS)))
        self.gate, self.up, self.down = gate, up, down
        self.norm_weight, self.activation, self.eps = norm_weight, activation, eps
        self.max_tokens = min(layer.max_tokens for layer in (gate, up, down))

        def rows(width, dtype=torch.bfloat16):
            return torch.empty(self.max_tokens, width, dtype=dtype, device=norm_weight.device)

        # the batch's intermediate rows; kept, so that a captured graph owns no others
        self.n, self.mid = rows(gate.K), rows(gate.N)
        self.nq = rows(gate.K, torch.float8_e4m3fn) if gate.fp8_base else None
        self.sn = rows(1, torch.float32).view(-1) if gate.fp8_base else None

    def forward(self, x: torch.Tensor, h: torch.Tensor, token_slot: torch.Tensor, y=None,
                residual: bool = False, stream=None) -> torch.Tensor:
        """x and the running residual ``h`` [T, hidden] (overwritten by h + x), and the rows' adapter
        slots.  Returns y, or h + y with ``residual`` (y may then be h, and else does not overlap it)."""
        T = x.shape[0]
        # (whatever can be refused is, before h changes; x and h by the norm)
        if T > self.max_tokens or token_slot.shape[0] < T:
            raise ValueError("more rows than max_tokens or than adapter slots")
        ids = token_slot[:T]
        if ids.dtype != torch.int32 or ids.device != x.device or ids.dim() != 1 or not ids.is_contiguous():
            raise ValueError("token_slot must be a dense int32 tensor on x's device")
        if residual and (h.data_ptr() % 16 or (h.dim() == 2 and T > 1 and h.stride(0) % 8)):
            raise ValueError("the rows of a residual must be 16-byte aligned")
        if y is None:
            y = empty(x.shape, x.dtype, x.device, stream)
        elif y.dtype != torch.bfloat16 or y.shape != (T, self.down.N) or y.device != x.device \
                or not y.is_contiguous() or y.data_ptr() % 16:
            raise ValueError("y must be a dense, 16-byte aligned bf16 tensor of x's shape on x's device")
        elif _overlap(y, h) and not (residual and y.data_ptr() == h.data_ptr() and h.is_contiguous()):
            raise ValueError("y and h overlap (y may be h itself in a pass with residual)")
        n, mid, nq, sn = self.n[:T], self.mid[:T], None, None
        if self.nq is not None:
            nq, sn = self.nq[:T], self.sn[:T]
        lora_rms_norm(x, self.norm_weight, self.eps, h, h, n, nq, sn, stream)
        for layer in (self.up, self.gate, self.down):
            layer.set_batch(ids, stream)
        _product(self.up, n, mid, nq, sn, stream)
        self.gate.forward_fused(n, mid, activation=self.activation, factor=mid, xq=nq, sx=sn,
                                stream=stream)
        if residual:
            return self.down.forward_fused(mid, y, residual=h, stream=stream)
        return _product(self.down, mid, y, None, None, stream)
