"""ctypes binding of the paged 4-bit key/value cache, the attention over it and a batch's block
tables and slot maps (``include/lora_kv.h``).

The functions carry the C names; they check what the C entry points cannot see (types, devices,
sizes and strides of the tensors) and raise ``LoraError`` with LORA_EINVAL, so that no
undersized tensor becomes an access out of bounds.  ``KvCache`` owns one cache, ``PageTable``
the pages of a set of requests.
"""
from __future__ import annotations

import ctypes

import torch

from .lora import LORA_EINVAL, LoraError, _stream, empty, library

_lib = library()
_I32, _BF16 = torch.int32, torch.bfloat16


def _bad(what: str):
    raise LoraError(LORA_EINVAL, what)


def _i32(name: str, t, n: int, device: int) -> int:
    """The address of a contiguous int32 tensor of at least n elements on the device."""
    if t.dtype is not _I32 or t.get_device() != device or not t.is_contiguous() or t.numel() < n:
        _bad("%s must be a contiguous int32 tensor of at least %d elements on the current CUDA "
             "device" % (name, n))
    return t.data_ptr()


def _rows(name: str, t, shape, device: int) -> int:
    """The row distance of a bf16 tensor [T, heads, dim] on the device whose rows are dense."""
    if t.dtype is not _BF16 or t.get_device() != device or t.shape != shape:
        _bad("%s must be a bf16 tensor of shape %s on the current CUDA device, not %s %s on %s"
             % (name, shape, t.dtype, tuple(t.shape), t.device))
    row, head, one = t.stride()
    if (shape[2] > 1 and one != 1) or (shape[1] > 1 and head != shape[2]):
        _bad("%s: the heads of a row must be dense" % name)
    width = shape[1] * shape[2]
    return row if shape[0] > 1 else max(row - row % 8, width)  # one row has no distance


def _check(rc: int, what: str) -> None:
    if rc < 0:
        raise LoraError(rc, what)


def lora_kv_maps(lens, new, adapter, page_size, block_table, free_pages, n_free, kv_len,
                 q_offsets, position, kv_slot, token_slot, counts, stream=None) -> None:
    """Block tables and slot maps of one batch (``lora_kv_maps``).  ``adapter`` may be None;
    the token arrays' length is T, ``block_table`` is [B, max_blocks]."""
    B, T, dev = lens.shape[0], kv_slot.shape[0], torch.cuda.current_device()
    if block_table.dim() != 2 or block_table.shape[0] < B:
        _bad("block_table must be [B, max_blocks]")
    rc = _lib.lora_kv_maps(
        _i32("lens", lens, B, dev), _i32("new", new, B, dev),
        None if adapter is None else _i32("adapter", adapter, B, dev), B, T, page_size,
        _i32("block_table", block_table, 1, dev), block_table.shape[1],
        _i32("free_pages", free_pages, 1, dev), free_pages.shape[0], _i32("n_free", n_free, 1, dev),
        _i32("kv_len", kv_len, B, dev), _i32("q_offsets", q_offsets, B + 1, dev),
        _i32("position", position, T, dev), _i32("kv_slot", kv_slot, T, dev),
        _i32("token_slot", token_slot, T, dev), _i32("counts", counts, 5, dev), _stream(stream, dev))
    _check(rc, "lora_kv_maps")


def lora_kv_release(done, lens, page_size, block_table, free_pages, n_free, status,
                    stream=None) -> None:
    """Return the pages of the requests with ``done[b] != 0`` (``lora_kv_release``)."""
    B, dev = lens.shape[0], torch.cuda.current_device()
    if block_table.dim() != 2 or block_table.shape[0] < B:
        _bad("block_table must be [B, max_blocks]")
    rc = _lib.lora_kv_release(
        _i32("done", done, B, dev), _i32("lens", lens, B, dev), B, page_size,
        _i32("block_table", block_table, 1, dev), block_table.shape[1],
        _i32("free_pages", free_pages, 1, dev), free_pages.shape[0], _i32("n_free", n_free, 1, dev),
        _i32("status", status, 1, dev), _stream(stream, dev))
    _check(rc, "lora_kv_release")


class PageTable:
    """The pages of up to ``max_requests`` requests and the maps of their current batch.

    ``step`` maps one batch of at most ``max_tokens`` new tokens: ``q_offsets``, ``kv_len``,
    ``position``, ``kv_slot`` and ``token_slot`` then describe it.  Everything stays on the
    GPU, and a step can be captured in a CUDA graph.
    """

    def __init__(self, num_pages: int, page_size: int, max_requests: int, max_blocks: int,
                 max_tokens: int, device="cuda"):
        def zeros(*n):
            return torch.zeros(*n, dtype=torch.int32, device=device)

        self.page_size, self.max_requests = page_size, max_requests
        self.block_table = zeros(max_requests, max_blocks)
        # pages leave the stack from its top: page 0 first
        self.free_pages = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.counts = zeros(5)
        self.counts[1] = num_pages
        self.n_free = self.counts[1:2]
        self.kv_len, self.q_offsets = zeros(max_requests), zeros(max_requests + 1)
        self.position, self.kv_slot = zeros(max_tokens), zeros(max_tokens)
        self.token_slot = zeros(max_tokens)
        self._status = zeros(1)

    def step(self, new, adapter=None, stream=None) -> None:
        """``new`` [max_requests] int32 (CUDA): tokens each request adds, 0 for idle ones;
        ``adapter`` their adapter slots."""
        lora_kv_maps(self.kv_len, new, adapter, self.page_size, self.block_table,
                     self.free_pages, self.n_free, self.kv_len, self.q_offsets, self.position,
                     self.kv_slot, self.token_slot, self.counts, stream)

    def release(self, done, stream=None) -> None:
        """The pages of requests with ``done[b] != 0`` are free again, their length 0."""
        lora_kv_release(done, self.kv_len, self.page_size, self.block_table, self.free_pages,
                        self.n_free, self._status, stream)

    def status(self):
        """(new tokens of the batch, free pages, pages taken, error flags of the last step and
        of the last release).  Synchronises."""
        c = self.counts.tolist()
        return c[0], c[1], c[2], c[3], int(self._status)


class KvCache:
    """Owns one 4-bit cache: ``num_pages`` pages of ``page_size`` positions for ``kv_heads``
    heads of ``head_dim`` dimensions (64 or 128)."""

    def __init__(self, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
                 max_requests: int, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
        self.handle = None
        h = ctypes.c_void_p()
        _check(_lib.lora_kv_cache_create(ctypes.byref(h), num_pages, page_size, kv_heads, head_dim,
                                         max_requests, k_scale, v_scale, _stream(stream)),
               "lora_kv_cache_create")
        self.handle = h.value
        self.num_pages, self.page_size = num_pages, page_size
        self.kv_heads, self.head_dim, self.max_requests = kv_heads, head_dim, max_requests

    def _check(self, rc: int) -> None:
        if rc < 0:
            raise LoraError(rc, _lib.lora_kv_last_error(self.handle).decode())

    def append(self, k, v, kv_slot, stream=None) -> None:
        """Write k and v [T, kv_heads, head_dim] (bf16; rows may be apart) to ``kv_slot`` [T]."""
        T, dev = k.shape[0], torch.cuda.current_device()
        shape = (T, self.kv_heads, self.head_dim)
        ldk, ldv = _rows("k", k, shape, dev), _rows("v", v, shape, dev)
        self._check(_lib.lora_kv_append(self.handle, k.data_ptr(), ldk, v.data_ptr(), ldv,
                                        _i32("kv_slot", kv_slot, T, dev), T, _stream(stream, dev)))

    def read(self, kv_slot, k_out=None, v_out=None, stream=None):
        """The values held in ``kv_slot`` [T], as bf16 [T, kv_heads, head_dim]."""
        T, dev = kv_slot.shape[0], torch.cuda.current_device()
        shape = (T, self.kv_heads, self.head_dim)
        if k_out is None:
            k_out = empty(shape, _BF16, kv_slot.device, stream)
        if v_out is None:
            v_out = empty(shape, _BF16, kv_slot.device, stream)
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            _rows(name, t, shape, dev)
            if not t.is_contiguous():
                _bad("%s must be contiguous" % name)
        self._check(_lib.lora_kv_read(self.handle, _i32("kv_slot", kv_slot, T, dev), T,
                                      k_out.data_ptr(), v_out.data_ptr(), _stream(stream, dev)))
        return k_out, v_out

    def attend(self, q, q_offsets, kv_len, block_table, max_q: int, scale: float = None, out=None,
               stream=None):
        """softmax(scale q K^T) V for q [T, q_heads, head_dim] (bf16; rows may be apart).
        ``scale`` is head_dim ** -0.5 by default; ``max_q`` bounds a request's query rows."""
        T, q_heads = q.shape[0], q.shape[1]
        B, dev = kv_len.shape[0], torch.cuda.current_device()
        shape = (T, q_heads, self.head_dim)
        if out is None:
            out = empty(shape, _BF16, q.device, stream)
        if block_table.dim() != 2 or block_table.shape[0] < B:
            _bad("block_table must be [B, max_blocks]")
        if scale is None:
            scale = self.head_dim ** -0.5
        self._check(_lib.lora_kv_attend(
            self.handle, q.data_ptr(), _rows("q", q, shape, dev), q_heads,
            _i32("q_offsets", q_offsets, B + 1, dev), _i32("kv_len", kv_len, B, dev),
            _i32("block_table", block_table, 1, dev), block_table.shape[1], B, T, max_q, scale,
            out.data_ptr(), _rows("out", out, shape, dev), _stream(stream, dev)))
        return out

    def status(self, stream=None) -> int:
        """LORA_OK, LORA_EID or LORA_ETIMEOUT since the last call (synchronises)."""
        return _lib.lora_kv_get_status(self.handle, _stream(stream))

    def wait_selftest(self, stream=None) -> None:
        """Leave the cache as a wait that ran out leaves it (``lora_kv_wait_selftest``): ``status``
        then returns LORA_ETIMEOUT, and the cache is usable again."""
        self._check(_lib.lora_kv_wait_selftest(self.handle, _stream(stream)))

    def nbytes(self) -> int:
        return int(_lib.lora_kv_cache_bytes(self.handle))

    def close(self):
        if getattr(self, "handle", None):
            _lib.lora_kv_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
