"""Mixed-adapter products with bias, activation, factor and residual in their epilogue, on the GPU,
against the CPU oracle's sums in 64 bits.

Tolerance.  The parity bar of a forward holds its fp32 sum within 2e-3 of the definition's (beside
the rounding to bf16, 2^-8 of the result).  That error passes the activation, whose slope is at most
1.13 (GELU; SiLU 1.1, ReLU 1), and is multiplied by the factor.  The activation's own error (an
exponential and a quotient of 2 units in the last place each, whose argument is off by a few 2^-24
of itself), the bias's, product's and residual's sums are within 2^-18 of the terms' sizes for
sums below 2^4, as these are.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from segmented_rank_gemm_gb300 import workloads

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _act(x, name):
    if name == "relu":
        return np.maximum(x, 0)
    if name == "gelu":
        return x * 0.5 * (1 + np.vectorize(math.erf)(x / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + np.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    if name == "silu":
        return x / (1 + np.exp(-x))
    return x


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, seed, T, K, N, S=6, ranks=(1, 16, 8, 3, 12, 2), R=16, e4m3=False, layout="random", **kw):
        from segmented_rank_gemm_gb300.lora import LoraLayer
        self.wl = wl = workloads.synthetic(seed, T, K, N, S=S, ranks=list(ranks)[:S], R=R, layout=layout, **kw)
        self.layer = LoraLayer(wl.W.cuda(), S, R, max(T, 1), fp8_base=e4m3)
        for s, ad in enumerate(wl.adapters):
            if ad is not None:
                self.layer.load(s, ad[0].cuda(), ad[1].cuda(), ad[2])
        table = oracle.SlotTable(wl.adapters, K, N)
        if e4m3:
            self.sums = fp8.base_w8a8(wl.x.float().numpy(), wl.W.float().numpy()) + oracle.forward_rows(
                wl.x, torch.zeros(K, N, dtype=torch.float64), table, wl.token_slot)
        else:
            self.sums = oracle.forward_rows(wl.x, wl.W, table, wl.token_slot)
        g = torch.Generator().manual_seed(seed)
        self.bias, self.factor, self.residual = (torch.randn(*n, generator=g).bfloat16()
                                                 for n in ((N,), (T, N), (T, N)))
        self.x, self.ids = wl.x.cuda(), wl.token_slot.cuda()

    def check(self, act, bias, factor, residual, /, y=None, what="", **more):
        self.layer.set_batch(self.ids)
        given = {n: t.cuda() if isinstance(t, torch.Tensor) else None for n, t in
                 (("bias", self.bias if bias else None), ("factor", self.factor if factor else None),
                  ("residual", self.residual if residual else None))}
        out = self.layer.forward_fused(self.x, y, activation=act, **{**given, **more})
        torch.cuda.synchronize()
        self.close(out, act, bias, factor, residual, what)
        return out

    def close(self, out, act, bias, factor, residual, what=""):
        v = self.sums + (_np(self.bias) if bias else 0)
        f = _np(self.factor) if factor else np.ones(1)
        r = _np(self.residual) if residual else np.zeros(1)
        a = _act(v, act)
        want = a * f + r
        lim = 2.0 ** -8 * np.abs(want) + 1.13 * 2e-3 * np.abs(f) + 2.0 ** -18 * (np.abs(a * f) + np.abs(r))
        got = _np(out)
        assert np.isfinite(got).all(), what
        over = np.abs(got - want) - lim
        assert (over <= 0).all(), "%s: %d over, by up to %.3g" % (what, (over > 0).sum(), over.max())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", [(1, 64, 72), (129, 256, 1040), (300, 512, 264), (600, 512, 264)])
def test_every_epilogue(T, K, N, act, e4m3):
    c = Case(40 + T, T, K, N, e4m3=e4m3, w_std=0.08, base_frac=0.2)
    for parts in range(8):
        c.check(act, parts & 1, parts & 2, parts & 4, what="%s parts %d" % (act, parts))
    assert c.layer.status() == 0
    c.layer.close()


def test_nothing_to_do_is_the_plain_forward():
    for T in (100, 700):
        for e4m3 in (False, True):
            c = Case(T, T, 256, 392, e4m3=e4m3)
            want = c.layer(c.x, c.ids)
            assert torch.equal(c.layer.forward_fused(c.x), want)
            assert torch.equal(c.layer.forward_fused(c.x, bias=torch.zeros(392, dtype=torch.bfloat16, device="cuda")),
                               want)
            c.layer.close()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [300, 1000])
def test_every_tiling(T, e4m3):
    c = Case(60, T, 1024, 520, S=5, ranks=[16] * 5, e4m3=e4m3, base_frac=0.1, layout="runs")
    for bn in (64, 128, 256):
        for ks in (1, 2, 4):
            for pair in (0, 1):
                if bn // ks < 32 or (pair and bn < 128) or (T > 512 and ks > 1):
                    continue
                c.layer.set_gemm_plan(bn, ks, pair)
                c.check("silu", True, True, True, what="plan (%d, %d, %d)" % (bn, ks, pair))
    assert c.layer.status() == 0
    c.layer.close()


@pytest.mark.parametrize("T,K,N,e4m3", [(512, 512, 14336, False), (512, 1024, 14336, True),
                                        (1200, 2048, 4104, False)])
def test_batches_of_two_launches_and_of_cut_tiles(T, K, N, e4m3):
    # the automatic plans that run a batch as two launches, or cut the last round's tiles in two
    c = Case(70, T, K, N, S=3, ranks=[16, 8, 4], e4m3=e4m3, base_frac=0.1, layout="runs")
    c.check("silu", True, True, True)
    y = c.residual.cuda()
    c.check("gelu", False, True, True, y=y, residual=y)
    c.layer.close()


def test_pooled_and_composed_adapters_and_wide_ranks():
    from segmented_rank_gemm_gb300.lora import LoraLayer
    for T in (200, 800):
        wl = workloads.synthetic(80, T, 256, 264, S=4, ranks=[64, 1, 33, 7], R=64, base_frac=0.1)
        c = Case(80, T, 256, 264, S=4, ranks=[64, 1, 33, 7], R=64, base_frac=0.1)
        c.check("silu", True, True, True)
        plain = c.layer
        c.layer = LoraLayer(wl.W.cuda(), 4, 64, T, pool_rows=128)
        for s, (A, B, alpha) in enumerate(wl.adapters):
            c.layer.load_composed(s, [(A.cuda(), B.cuda(), alpha, 1.0)])
        c.check("silu", True, True, True)
        c.layer.close()
        plain.close()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("R", [8, 32, 40, 64, 72, 128])
def test_every_width_of_slots(R, e4m3):
    # the ring and what lies beside it in shared memory change with the slots' width
    for T, N in ((64, 328), (700, 2056), (2300, 4104)):
        c = Case(85, T, 256, N, S=3, ranks=[R, 1, max(1, R // 2)], R=R, e4m3=e4m3, base_frac=0.1, layout="runs")
        for parts in ((1, 1, 1), (0, 1, 0), (0, 0, 1)):
            c.check("silu", *parts, what="R=%d T=%d" % (R, T))
        assert c.layer.status() == 0
        c.layer.close()


def test_strided_rows_in_place_and_nothing_beside():
    c = Case(90, 150, 256, 264)
    N, wide = 264, torch.full((150, 2 * 264 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    f, r = wide[:, 8:8 + N], wide[:, 16 + N:16 + 2 * N]
    f.copy_(c.factor)
    r.copy_(c.residual)
    c.check("gelu", True, True, True, factor=f, residual=r)
    for in_place in ("factor", "residual"):
        y = getattr(c, in_place).cuda()
        out = c.check("silu", True, True, True, y=y, **{in_place: y})
        assert out.data_ptr() == y.data_ptr()
    # rows of a larger array: what lies behind them is not written
    big = torch.full((160, N), 3.0, dtype=torch.bfloat16, device="cuda")
    c.check("none", False, False, True, y=big[:150])
    assert (big[150:] == 3).all()
    c.layer.close()


def test_given_e4m3_rows():
    from segmented_rank_gemm_gb300.norm import rms_norm
    for T in (64, 700):
        c = Case(95, T, 512, 256, e4m3=True)
        w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
        xq = torch.empty(T, 512, dtype=torch.float8_e4m3fn, device="cuda")
        sx = torch.empty(T, device="cuda")
        x = rms_norm(c.x, w, xq=xq, sx=sx)
        c.layer.set_batch(c.ids)
        plain = c.layer.forward_e4m3(x, xq, sx)
        assert torch.equal(c.layer.forward_fused(x, xq=xq, sx=sx), plain)
        # (a step of bf16 about the rounded sum, 2^-8 of it to both sides, is multiplied by two)
        two = torch.full((T, 256), 2.0, dtype=torch.bfloat16, device="cuda")
        assert torch.equal(c.layer.forward_fused(x, factor=two, xq=xq, sx=sx), plain * 2)
        c.layer.close()


@pytest.mark.parametrize("act", ACTS)
def test_large_and_unbounded_sums(act):
    # far tails of the activations, infinities and NaN in a bias: they stay in their columns
    c = Case(97, 40, 64, 64, w_std=0.02)
    big = [0.0, 3e38, -3e38, 100.0, -100.0, 40.0, -40.0, 12.0, -12.0, 5.0, -5.0, 1e-30]
    c.bias[:len(big)] = torch.tensor(big).bfloat16()
    c.layer.set_batch(c.ids)
    out = _np(c.layer.forward_fused(c.x, bias=c.bias.cuda(), activation=act))
    with np.errstate(over="ignore"):
        v = c.sums + _np(c.bias)
        want = _act(v, act)
    # (x^3 of 3e38 overflows in fp32: the approximation's tanh is 1 there all the same)
    lim = 2.0 ** -8 * np.abs(want) + 1.13 * 2e-3 + 2.0 ** -18 * np.abs(want)
    assert (np.abs(out - want) <= lim).all()
    for bad in (float("nan"), float("inf"), float("-inf")):
        b = c.bias.clone()
        b[20] = bad
        got = _np(c.layer.forward_fused(c.x, bias=b.cuda(), activation=act))
        if math.isnan(bad):
            assert np.isnan(got[:, 20]).all()
        keep = np.arange(64) != 20
        assert np.array_equal(got[:, keep], out[:, keep])
    c.layer.close()


def test_streams_graphs_and_calls_in_a_row():
    c = Case(98, 256, 512, 512, S=4, ranks=[8, 16, 4, 2])
    f, r, b = c.factor.cuda(), c.residual.cuda(), c.bias.cuda()
    want = c.check("silu", True, True, True)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    y = torch.zeros_like(want)
    torch.cuda.synchronize()
    c.layer.set_batch(c.ids, stream)
    c.layer.forward_fused(c.x, y, bias=b, activation="silu", factor=f, residual=r, stream=stream)
    stream.synchronize()
    assert torch.equal(y, want)
    with torch.cuda.graph(graph):
        c.layer.set_batch(c.ids)
        c.layer.forward_fused(c.x, y, bias=b, activation="silu", factor=f, residual=r)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    # a residual that the call before writes, over and over
    h = r.clone()
    for _ in range(4):
        c.layer.set_batch(c.ids)
        c.layer.forward_fused(c.x, h, residual=h)
    ref = r.clone()
    for _ in range(4):
        c.layer.set_batch(c.ids)
        ref = c.layer.forward_fused(c.x, residual=ref)
        torch.cuda.synchronize()
    assert torch.equal(h, ref)
    c.layer.close()


def test_refusals():
    from segmented_rank_gemm_gb300.lora import Epilogue, LoraError, LoraLayer, lora_forward_fused
    c = Case(99, 20, 64, 64)
    f, b, y = c.factor.cuda(), c.bias.cuda(), torch.empty(20, 64, dtype=torch.bfloat16, device="cuda")
    c.layer.set_batch(c.ids)
    for bad in (dict(activation="tanh"), dict(factor=f[:19]), dict(factor=f.float()), dict(residual=f.t()[:20]),
                dict(bias=b[:60]), dict(bias=b.cpu()), dict(xq=f), dict(sx=b.float()), dict(residual=f[:, :56]),
                dict(xq=torch.zeros(20, 64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            c.layer.forward_fused(c.x, **bad)
    wide = torch.zeros(21, 68, dtype=torch.bfloat16, device="cuda")
    flat = torch.zeros(22 * 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(factor=wide[:20, :64]), dict(residual=flat[4:4 + 20 * 64].view(20, 64)),
                dict(y=flat[:20 * 64].view(20, 64), residual=flat[64:21 * 64].view(20, 64)),
                dict(y=flat[:20 * 64].view(20, 64), bias=flat[64:128]),
                dict(xq=torch.zeros(20, 64, dtype=torch.uint8, device="cuda"), sx=torch.ones(20, device="cuda"))):
        with pytest.raises(LoraError):
            c.layer.forward_fused(c.x, **bad)
    for ep in (Epilogue(activation=5), Epilogue(activation=-1), Epilogue(factor=f.data_ptr(), ldf=56),
               Epilogue(residual=f.data_ptr(), ldr=68)):
        with pytest.raises(LoraError):
            lora_forward_fused(c.layer.handle, c.x, y, 20, ep)
    with pytest.raises(LoraError):  # not the batch's rows
        c.layer.forward_fused(c.x[:10])
    plain = LoraLayer(torch.zeros(64, 64, device="cuda"), 2, 8, 16)
    with pytest.raises(ValueError):
        plain.forward_fused(torch.zeros(4, 64, device="cuda"))
    plain.set_batch(c.ids[:4])
    with pytest.raises(LoraError):
        lora_forward_fused(plain.handle, torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, device="cuda"), 4,
                           Epilogue())
    c.check("none", True, True, True)
    c.layer.set_batch(c.ids[:0])
    assert c.layer.forward_fused(c.x[:0], residual=f[:0]).shape == (0, 64)
    assert c.layer.status() == 0
    c.layer.close()
    plain.close()
