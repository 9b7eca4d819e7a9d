"""Values that a fused forward's epilogue meets at its borders: sums that are infinite or NaN, and the far
tails of the activations, against the definitions in 64 bits.

The rows of x are zeros here, so that the sum before the activation is the bias, exactly.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
BF16, DEV = torch.bfloat16, "cuda"


def _act(v, name):
    """include/lora_layer.h's definitions, each operation in 64 bits."""
    if math.isnan(v):
        return v
    if name == "relu":
        return max(v, 0.0)
    if name == "gelu":
        return v * (1 + math.erf(v / math.sqrt(2))) / 2
    if name == "gelu_tanh":
        return v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))) / 2
    if name == "silu":
        return v / (1 + math.exp(-v)) if v > -700 else (math.nan if v == -math.inf else 0.0)
    return v


# decode (the delta mode's epilogue), prefill (the one of batches beyond 512 rows), and both over an e4m3 base
LAYERS = [(40, False), (600, False), (40, True), (600, True)]


def _layer(T, e4m3, N):
    from segmented_rank_gemm_gb300.lora import LoraLayer
    layer = LoraLayer(torch.ones(64, N, dtype=BF16, device=DEV), 2, 8, T, fp8_base=e4m3)
    layer.set_batch(torch.full((T,), -1, dtype=torch.int32, device=DEV))
    return layer, torch.zeros(T, 64, dtype=BF16, device=DEV)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,e4m3", LAYERS)
def test_infinite_and_nan_sums(T, e4m3, act):
    sums = [math.inf, -math.inf, math.nan, 3e38, -3e38, 1.0, 0.0]
    layer, x = _layer(T, e4m3, 64)
    bias = torch.zeros(64, dtype=BF16, device=DEV)
    bias[8:8 + len(sums)] = torch.tensor(sums).to(BF16).to(DEV)
    want = [_act(v, act) if abs(v) < 1e38 or not math.isfinite(v) else
            {"none": v, "relu": max(v, 0.0)}.get(act, v if v > 0 else 0.0) for v in sums]
    for f in (None, 2.0, -1.0):
        factor = None if f is None else torch.full((T, 64), f, dtype=BF16, device=DEV)
        y = layer.forward_fused(x, bias=bias, activation=act, factor=factor).double().cpu().numpy()
        for i, (v, w) in enumerate(zip(sums, want)):
            with np.errstate(over="ignore", invalid="ignore"):
                w = float(torch.tensor(w * (1 if f is None else f)).to(BF16))  # (6e38 is an infinity)
            got = y[:, 8 + i]
            if math.isnan(w):
                assert np.isnan(got).all(), (act, v, f, got[0])
            elif math.isinf(w):
                assert (got == w).all(), (act, v, f, got[0])
            else:
                assert (np.abs(got - w) <= 2.0 ** -8 * abs(w)).all(), (act, v, f, got[0])
    layer.close()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,e4m3", LAYERS)
def test_tails_of_the_activations(T, e4m3, act):
    # One rounding of the result (2^-8 of it); the exponent's error (up to 126, rounded by some four
    # operations in fp32: 4 2^-24 126 ln 2 < 2^-15, with the exponential's and the reciprocal's own below
    # 2^-14 of the result); and what is lost where an exponential or a reciprocal falls below 2^-126 and
    # counts as 0: at most 2^-126 of the sum.  (bf16 holds 2^-133.)
    v = torch.cat((torch.linspace(-14, 14, 1024), torch.linspace(-100, 100, 1024))).to(BF16)
    layer, x = _layer(T, e4m3, len(v))
    got = layer.forward_fused(x, bias=v.to(DEV), activation=act).double().cpu().numpy()
    v = v.double().numpy()
    want = np.array([_act(float(t), act) for t in v])
    if act == "gelu":  # (1 + erf cancels in 64 bits: the same by erfc)
        want = np.array([t * math.erfc(-t / math.sqrt(2)) / 2 for t in v])
    if act == "gelu_tanh":  # the same, without its cancellation: t / (1 + e^-2u)
        u = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        want = v / (1 + np.exp(np.minimum(-2 * u, 700)))
    lim = (2.0 ** -8 + 2.0 ** -14) * np.abs(want) + 2.0 ** -126 * np.maximum(np.abs(v), 1)
    assert (np.abs(got - want) <= lim).all(), float((np.abs(got - want) / lim).max())
    layer.close()
