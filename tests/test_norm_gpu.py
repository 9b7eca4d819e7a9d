"""The residual norm on the GPU against its 64-bit definition.

Tolerances.  h is the fp32 sum rounded once: exact.  y is a product of fp32 values, each step
within 2^-24, and a sum of squares whose terms are all positive: the fp32 value is within 2^-20
relative of the exact one, and an output lies between the roundings of the exact value's two
neighbours at that distance.  Row scales likewise.  An e4m3 value is within half its step of y / sx, the step being 2^-3 of the value's
power of two and at least 2^-9, widened by 1e-5 for the quotient's own error.
"""
import numpy as np
import pytest
import torch

from oracle import kv as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _np(t):
    return t.detach().float().cpu().numpy()


def _inputs(T, K, dtype, residual=True, pad=0, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)

    def rows(s):
        return (torch.randn(T, K + pad, generator=g) * s).to(dtype).to(DEV)[:, :K]

    w = (1 + 0.2 * torch.randn(K, generator=g)).to(dtype).to(DEV)
    return rows(spread), rows(3 * spread) if residual else None, w


def _check(x, r, w, eps, h, y, xq, sx):
    h64, y64, s64 = ref.rms_norm(_np(x), None if r is None else _np(r), _np(w), eps)
    if h is not None:
        h32 = _np(x) + (0 if r is None else _np(r))
        assert torch.equal(h.cpu(), torch.from_numpy(h32).to(x.dtype))
    if y is not None:
        near, far = (_np(torch.from_numpy(np.abs(y64) * (1 + e)).to(x.dtype))
                     for e in (-2.0 ** -20, 2.0 ** -20))
        assert ((near <= np.abs(_np(y))) & (np.abs(_np(y)) <= far)).all()
        assert (_np(y) * y64 >= 0).all()
    if xq is not None:
        s = _np(sx).astype(np.float64)
        assert (np.abs(s - s64) <= 2.0 ** -20 * s64).all()
        v, t = np.abs(_np(xq).astype(np.float64)), np.abs(y64) / s[:, None]
        step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(t, 2.0 ** -6))) - 3), 2.0 ** -9)
        assert (np.abs(v - np.minimum(t, 448)) <= step / 2 + 1e-5 * t).all()
        assert (np.sign(_np(xq)) * np.sign(y64) >= 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 4096), (3, 7), (5, 8), (130, 64), (33, 257), (17, 1000),
                                 (9, 1024), (4, 1028), (6, 2056), (65, 4096), (3, 4097), (2, 8192),
                                 (2, 14336), (3, 16384), (2, 32768), (2, 32767)])
def test_norm(T, K, dtype):
    x, r, w = _inputs(T, K, dtype, seed=T + K)
    y, h = torch.empty_like(x), torch.empty_like(x)
    xq = torch.empty(T, K, dtype=torch.float8_e4m3fn, device=DEV)
    sx = torch.empty(T, device=DEV)
    from segmented_rank_gemm_gb300.norm import lora_rms_norm
    lora_rms_norm(x, w, 1e-6, r, h, y, xq, sx)
    _check(x, r, w, 1e-6, h, y, xq, sx)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [1, 8])
def test_strided_rows_and_in_place_residual(dtype, pad):
    from segmented_rank_gemm_gb300.norm import lora_rms_norm, rms_norm
    T, K = 20, 512
    x, r, w = _inputs(T, K, dtype, pad=pad, seed=pad)
    before = r.clone()
    y = rms_norm(x, w, 1e-5, residual=r, residual_out=r)
    _check(x, before, w, 1e-5, r, y, None, None)
    assert rms_norm(x, w, 1e-5).shape == (T, K)
    # h into x itself, without y
    x2 = x.clone()
    full = torch.zeros(T, 2 * K, dtype=dtype, device=DEV)
    full[:, :K] = x2
    lora_rms_norm(full[:, :K], w, 1e-5, before, full[:, :K])
    assert torch.equal(full[:, :K].cpu(), torch.from_numpy(_np(x2) + _np(before)).to(dtype))
    # h beside x in one buffer
    full[:, :K] = x2
    lora_rms_norm(full[:, :K], w, 1e-5, before, full[:, K:])
    assert torch.equal(full[:, K:].cpu(), torch.from_numpy(_np(x2) + _np(before)).to(dtype))


def test_special_rows():
    from segmented_rank_gemm_gb300.norm import lora_rms_norm
    T, K = 6, 264
    x, _, w = _inputs(T, K, torch.bfloat16, residual=False)
    x[0] = 0
    x[1] = 1e-20   # below eps
    x[2, 5] = float("nan")
    x[3] *= 1e15   # squares within fp32
    y = torch.empty_like(x)
    xq = torch.empty(T, K, dtype=torch.float8_e4m3fn, device=DEV)
    sx = torch.empty(T, device=DEV)
    lora_rms_norm(x, w, 1e-6, y=y, xq=xq, sx=sx)
    assert not y[0].any() and not _np(xq[0]).any() and float(sx[0]) == 1.0
    assert torch.isnan(y[2]).all()
    keep = [1, 3, 4, 5]
    _check(x[keep], None, w, 1e-6, None, y[keep], xq[keep], sx[keep])
    # eps 0 and a zero row: 0 / 0 by the definition
    lora_rms_norm(x, w, 0.0, y=y)
    assert torch.isnan(y[0]).all()


def test_many_rows_on_a_stream_and_in_a_graph():
    from segmented_rank_gemm_gb300.norm import rms_norm
    T, K = 3000, 1024
    x, r, w = _inputs(T, K, torch.bfloat16)
    y, h = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    rms_norm(x, w, residual=r, residual_out=h, y=y, stream=s)
    s.synchronize()
    _check(x, r, w, 1e-6, h, y, None, None)
    y2 = torch.empty_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rms_norm(x, w, residual=r, residual_out=h, y=y2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


def test_refusals():
    from segmented_rank_gemm_gb300.lora import LoraError
    from segmented_rank_gemm_gb300.norm import lora_rms_norm
    T, K = 4, 64
    x, r, w = _inputs(T, K, torch.bfloat16)
    y, sx = torch.empty_like(x), torch.empty(T, device=DEV)
    xq = torch.empty(T, K, dtype=torch.float8_e4m3fn, device=DEV)
    ok = dict(x=x, weight=w, eps=1e-6, residual=r, y=y)
    wide = torch.zeros(1, 32769, dtype=torch.bfloat16, device=DEV)
    for change in (dict(x=x.half()), dict(x=x.cpu()), dict(weight=w[:-1]), dict(weight=w.float()),
                   dict(residual=r[:2]), dict(y=y[:2]), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(xq=xq), dict(sx=sx), dict(y=None), dict(y=x), dict(y=r), dict(x=x.t()),
                   dict(residual_out=y), dict(xq=xq[:2], sx=sx), dict(xq=xq, sx=sx[:2]),
                   dict(residual_out=r[:, :32]),
                   dict(x=wide, weight=wide[0], residual=None, y=torch.empty_like(wide))):
        with pytest.raises(LoraError):
            lora_rms_norm(**{**ok, **change})
    lora_rms_norm(**ok)
    lora_rms_norm(x[:0], w, 1e-6, y=y[:0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(7, 2), (5, 127), (6, 130), (3, 511), (4, 512), (5, 514), (4, 1026), (3, 2047),
                                 (2, 2050), (3, 4090), (2, 4095), (2, 8190), (2, 12000), (2, 16384), (2, 16386),
                                 (1, 32766), (3, 24576)])
def test_norm_at_every_split(T, K, dtype):
    # widths on both sides of the splits of rows of vectors, pairs and elements
    x, r, w = _inputs(T, K, dtype, seed=T * K)
    y, h = torch.empty_like(x), torch.empty_like(x)
    xq = torch.empty(T, K, dtype=torch.float8_e4m3fn, device=DEV)
    sx = torch.empty(T, device=DEV)
    from segmented_rank_gemm_gb300.norm import lora_rms_norm
    lora_rms_norm(x, w, 1e-5, r, h, y, xq, sx)
    _check(x, r, w, 1e-5, h, y, xq, sx)


def test_norm_refuses_split_elements():
    from segmented_rank_gemm_gb300 import lora
    lib = lora.library()
    x, r, w = _inputs(4, 64, torch.bfloat16)
    y, sx = torch.empty_like(x), torch.empty(4, device=DEV)
    xq = torch.empty(4, 64, dtype=torch.float8_e4m3fn, device=DEV)
    good = [x.data_ptr(), 64, r.data_ptr(), 64, w.data_ptr(), 1e-6, 3, 63, lora.LORA_BF16, None, 0,
            y.data_ptr(), xq.data_ptr(), sx.data_ptr(), 0]
    for i in (0, 2, 4, 11, 13):
        bad = list(good)
        bad[i] += 1
        assert lib.lora_rms_norm(*bad) == lora.LORA_EINVAL
    assert lib.lora_rms_norm(*good) == 0
    torch.cuda.synchronize()
