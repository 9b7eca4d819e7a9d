"""ctypes binding of the paged 4-bit key/value cache, the rotation and the attentions over it and a
batch's block tables and slot maps (``include/lora_kv.h``).

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
    if t.is_contiguous():
        return shape[1] * shape[2]
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


def lora_kv_release_shared(done, lens, shared, page_size, block_table, free_pages, n_free, status,
                           stream=None) -> None:
    """``lora_kv_release`` of requests whose first ``shared[b]`` positions are another's
    (``lora_kv_release_shared``)."""
    B, dev = lens.shape[0], torch.cuda.current_device()
    if block_table.dim() != 2 or block_table.shape[0] < B:
        _bad("block_table must be [B, max_blocks]")
    rc = _lib.lora_kv_release_shared(
        _i32("done", done, B, dev), _i32("lens", lens, B, dev), _i32("shared", shared, B, dev), B,
        page_size, _i32("block_table", block_table, 1, dev), block_table.shape[1],
        _i32("free_pages", free_pages, 1, dev), free_pages.shape[0], _i32("n_free", n_free, 1, dev),
        _i32("status", status, 1, dev), _stream(stream, dev))
    _check(rc, "lora_kv_release_shared")


def lora_kv_fork(parent, want, lens, shared, page_size, block_table, status, stream=None) -> None:
    """Requests that start with the whole pages of ``parent[b]`` (-1: unchanged), up to ``want[b]``
    positions if given (``lora_kv_fork``)."""
    B, dev = lens.shape[0], torch.cuda.current_device()
    if block_table.dim() != 2 or block_table.shape[0] < B:
        _bad("block_table must be [B, max_blocks]")
    rc = _lib.lora_kv_fork(
        _i32("parent", parent, B, dev), None if want is None else _i32("want", want, B, dev),
        _i32("lens", lens, B, dev), _i32("shared", shared, B, dev), B, page_size,
        _i32("block_table", block_table, 1, dev), block_table.shape[1],
        _i32("status", status, 1, dev), _stream(stream, dev))
    _check(rc, "lora_kv_fork")


def _ready(t) -> None:
    """What an object's constructor enqueued is done: a call on any stream may be its first."""
    if t.is_cuda:
        torch.cuda.current_stream(t.device).synchronize()


class Rotary:
    """The angles of a rotation of queries and keys by position, for ``KvCache.append_rotated``:
    ``angles`` [max_position, 2, rotary_dim / 2] fp32, the cosines and sines, computed in 64 bits, of
    p * frequency[i].  The first ``rotary_dim`` dimensions of a head are turned, a multiple of 32:
    pair i is dimensions i and i + rotary_dim / 2, or 2 i and 2 i + 1 if ``interleaved``.
    ``frequencies`` [rotary_dim / 2] default to theta ** (-2 i / rotary_dim)."""

    def __init__(self, max_position: int, rotary_dim: int, theta: float = 10000.0,
                 interleaved: bool = False, frequencies=None, device="cuda"):
        if max_position < 1 or rotary_dim < 32 or rotary_dim % 32:
            raise ValueError("max_position must be positive, rotary_dim a multiple of 32")
        if frequencies is None:
            i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
            frequencies = theta ** (-2 * i / rotary_dim)
        elif tuple(frequencies.shape) != (rotary_dim // 2,):
            raise ValueError("frequencies must be [rotary_dim / 2]")
        angle = torch.outer(torch.arange(max_position, dtype=torch.float64, device=device),
                            frequencies.to(device=device, dtype=torch.float64))
        self._angles = torch.stack((angle.cos(), angle.sin()), 1).float().contiguous()
        _ready(self._angles)
        self.max_position, self.rotary_dim, self.interleaved = max_position, rotary_dim, interleaved

    @property
    def angles(self) -> torch.Tensor:
        return self._angles


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
        self.shared_len = zeros(max_requests)  # positions that are another request's pages
        self._status, self._fork_status = zeros(1), zeros(1)
        _ready(self.free_pages)

    def step(self, new, adapter=None, stream=None) -> None:
        """``new`` [max_requests] int32 (CUDA): tokens each request adds, 0 for idle ones;
        ``adapter`` their adapter slots."""
        lora_kv_maps(self.kv_len, new, adapter, self.page_size, self.block_table,
                     self.free_pages, self.n_free, self.kv_len, self.q_offsets, self.position,
                     self.kv_slot, self.token_slot, self.counts, stream)

    def fork(self, parent, want=None, stream=None) -> None:
        """Request b starts with the whole pages of request ``parent[b]`` (-1: unchanged), up to
        ``want[b]`` positions if given; it must be empty.  ``shared_len`` then says how many
        positions that are.  The pages stay the parent's, which is released with it or later."""
        lora_kv_fork(parent, want, self.kv_len, self.shared_len, self.page_size, self.block_table,
                     self._fork_status, stream)

    def fork_status(self) -> int:
        """Error flags of the last fork (which then changed nothing).  Synchronises."""
        return int(self._fork_status)

    def release(self, done, stream=None) -> None:
        """The pages of requests with ``done[b] != 0`` (but for those that are another's) are free
        again, their length 0; nothing changes where one that stays shares them (``status``: 4)."""
        lora_kv_release_shared(done, self.kv_len, self.shared_len, self.page_size,
                               self.block_table, self.free_pages, self.n_free, self._status, stream)

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

    def append_rotated(self, q, k, v, position, kv_slot, rotary: Rotary, q_out=None, stream=None):
        """``append`` with q [T, q_heads, head_dim] and k turned by ``position`` [T] first
        (``rotary``: a ``Rotary``).  The turned queries go to ``q_out`` (which may be q; a new
        tensor if not given), which is returned; k itself stays as it is."""
        T, q_heads, dev = q.shape[0], q.shape[1], torch.cuda.current_device()
        shape, q_shape = (T, self.kv_heads, self.head_dim), (T, q_heads, self.head_dim)
        ldq, ldk, ldv = _rows("q", q, q_shape, dev), _rows("k", k, shape, dev), _rows("v", v, shape, dev)
        angles = rotary._angles  # (of its own making: the device is all that can be wrong)
        if angles.get_device() != dev:
            _bad("the angles must be on the current CUDA device")
        # (names of their own: a tensor that only the caller's expression held would be freed here, and
        # its memory could become q_out's)
        position_at, slot_at = _i32("position", position, T, dev), _i32("kv_slot", kv_slot, T, dev)
        if q_out is None:
            q_out = empty(q_shape, _BF16, q.device, stream)
        self._check(_lib.lora_kv_append_rotated(
            self.handle, q.data_ptr(), ldq, q_heads, q_out.data_ptr(), _rows("q_out", q_out, q_shape, dev),
            k.data_ptr(), ldk, v.data_ptr(), ldv, position_at, slot_at, T, angles.data_ptr(),
            rotary.max_position, rotary.rotary_dim, rotary.interleaved, _stream(stream, dev)))
        return q_out

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

    def _attend(self, call, q, q_offsets, kv_len, block_table, max_q, scale, out, stream, more=()):
        """One of the attention entry points; ``more`` are its arguments behind max_q."""
        T, q_heads = q.shape[0], q.shape[1]
        B, dev = kv_len.shape[0], torch.cuda.current_device()
        shape = (T, q_heads, self.head_dim)
        if out is None:
            out = empty(shape, _BF16, q.device, stream)
        if block_table.dim() != 2 or block_table.shape[0] < B:
            _bad("block_table must be [B, max_blocks]")
        if scale is None:
            scale = self.head_dim ** -0.5
        before, behind = more if more else ((), ())
        self._check(call(
            self.handle, q.data_ptr(), _rows("q", q, shape, dev), q_heads,
            _i32("q_offsets", q_offsets, B + 1, dev), _i32("kv_len", kv_len, B, dev),
            _i32("block_table", block_table, 1, dev), block_table.shape[1], B, T, max_q, *before, scale,
            out.data_ptr(), _rows("out", out, shape, dev), *behind, _stream(stream, dev)))
        return out

    def attend(self, q, q_offsets, kv_len, block_table, max_q: int, scale: float = None, out=None,
               stream=None, causal: bool = True):
        """softmax(scale q K^T) V for q [T, q_heads, head_dim] (bf16; rows may be apart).
        ``scale`` is head_dim ** -0.5 by default; ``max_q`` bounds a request's query rows.
        Without ``causal`` every row sees all that its request has cached, an encoder's states say
        (``lora_kv_attend_cross``)."""
        return self._attend(_lib.lora_kv_attend if causal else _lib.lora_kv_attend_cross, q, q_offsets,
                            kv_len, block_table, max_q, scale, out, stream)

    def shared_workspace(self, tokens: int, q_heads: int):
        """What ``attend_shared`` needs for ``tokens`` rows, to be kept from call to call (calls
        that may run at the same time need one each)."""
        n = _lib.lora_kv_shared_workspace(self.handle, tokens, q_heads)
        if n < 0:
            _bad("tokens=%d, q_heads=%d" % (tokens, q_heads))
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    @staticmethod
    def check_groups(requests: int, group_offsets, prefix_row=None, prefix_len=None):
        """Refuses groups that ``attend_shared`` would for so many requests (the tensors themselves: what
        they hold is checked on the GPU).  Their addresses, and their number."""
        dev = torch.cuda.current_device()
        if prefix_row is None or prefix_len is None:
            _bad("groups are group_offsets, prefix_row and prefix_len")
        groups = group_offsets.numel() - 1
        if not 1 <= groups <= requests:
            _bad("%d groups of %d requests" % (groups, requests))
        return (_i32("group_offsets", group_offsets, 2, dev), _i32("prefix_row", prefix_row, groups, dev),
                _i32("prefix_len", prefix_len, groups, dev), groups)

    def attend_shared(self, q, q_offsets, kv_len, block_table, max_q: int, group_offsets, prefix_row,
                      prefix_len, shared_len, scale: float = None, out=None, workspace=None,
                      stream=None):
        """``attend`` for requests that share prefixes by groups, each prefix read once for all of
        its group (``lora_kv_attend_shared``): group g is requests ``group_offsets[g]`` ..
        ``group_offsets[g + 1] - 1``; the first ``shared_len[b]`` positions of a member are
        ``prefix_len[g]`` (whole pages, those in row ``prefix_row[g]`` of the table), or 0: it is
        attended by itself."""
        B, dev = kv_len.shape[0], torch.cuda.current_device()
        before = (*self.check_groups(B, group_offsets, prefix_row, prefix_len),
                  _i32("shared_len", shared_len, B, dev))
        if workspace is None:
            n = _lib.lora_kv_shared_workspace(self.handle, q.shape[0], q.shape[1])
            workspace = empty((max(n, 0),), torch.uint8, q.device, stream)
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _bad("workspace must be a contiguous tensor on the current CUDA device")
        return self._attend(_lib.lora_kv_attend_shared, q, q_offsets, kv_len, block_table, max_q, scale,
                            out, stream,
                            (before, (workspace.data_ptr(), workspace.numel() * workspace.element_size())))

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
