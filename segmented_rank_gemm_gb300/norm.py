"""ctypes binding of the root-mean-square norm with the residual's addition
(``include/lora_norm.h``)."""
from __future__ import annotations

import torch

from .lora import LORA_BF16, LORA_EINVAL, LORA_F32, LoraError, _stream, empty, library

_lib = library()
_DTYPES = {torch.bfloat16: LORA_BF16, torch.float32: LORA_F32}


def _bad(what: str):
    raise LoraError(LORA_EINVAL, what)


def _rows(name: str, t, dtype, shape, device: int) -> int:
    """The row distance of a tensor [T, K] on the device whose rows are dense."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        _bad("%s must be a tensor of x's type and shape on the current CUDA device" % name)
    row, one = t.stride()
    T, K = shape
    if K > 1 and one != 1:
        _bad("%s: the elements of a row must be dense" % name)
    return row if T > 1 else max(row, K)  # one row has no distance


def _dense(name: str, t, dtype, shape, device: int) -> int:
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape \
            or not t.is_contiguous():
        _bad("%s must be a contiguous tensor %s of %s on the current CUDA device"
             % (name, shape, dtype))
    return t.data_ptr()


def lora_rms_norm(x, weight, eps, residual=None, residual_out=None, y=None, xq=None, sx=None,
                  stream=None) -> None:
    """h = x + residual; y = h rsqrt(mean(h^2) + eps) weight over the rows of x [T, K] (bf16 or
    fp32).  Outputs, each optional: ``residual_out`` (h; may be ``residual``), ``y``, and
    ``xq`` (float8_e4m3fn) with its row scales ``sx`` [T] (fp32)."""
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2 or dtype not in _DTYPES:
        _bad("x must be a CUDA tensor [T, K] of bf16 or fp32")
    (T, K), dev = shape, torch.cuda.current_device()
    ldx = _rows("x", x, dtype, shape, dev)
    ldr = _rows("residual", residual, dtype, shape, dev) if residual is not None else 0
    ldh = _rows("residual_out", residual_out, dtype, shape, dev) if residual_out is not None else 0
    rc = _lib.lora_rms_norm(
        x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
        _dense("weight", weight, dtype, (K,), dev), eps, T, K, _DTYPES[dtype],
        None if residual_out is None else residual_out.data_ptr(), ldh,
        None if y is None else _dense("y", y, dtype, shape, dev),
        None if xq is None else _dense("xq", xq, torch.float8_e4m3fn, shape, dev),
        None if sx is None else _dense("sx", sx, torch.float32, (T,), dev), _stream(stream, dev))
    if rc < 0:
        raise LoraError(rc, "lora_rms_norm")


def rms_norm(x, weight, eps=1e-6, residual=None, residual_out=None, y=None, xq=None, sx=None,
             stream=None):
    """``lora_rms_norm`` returning y; ``y`` is allocated if not given."""
    if y is None:
        y = empty(x.shape, x.dtype, x.device, stream)
    lora_rms_norm(x, weight, eps, residual, residual_out, y, xq, sx, stream)
    return y
