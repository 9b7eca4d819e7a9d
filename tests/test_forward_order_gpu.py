"""Forwards of more than 512 rows right behind the kernel that writes their rows, the batch having
been set before it: the base product reads what that kernel wrote."""
import pytest
import torch

from segmented_rank_gemm_gb300 import workloads
from gpu_helpers import assert_parity, oracle_rows

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def _layer(wl, fp8_base=False):
    from segmented_rank_gemm_gb300.lora import LoraLayer
    layer = LoraLayer(wl.W.to(DEV), wl.S, wl.R, wl.T, fp8_base=fp8_base)
    for s, (A, B, alpha) in enumerate(wl.adapters):
        layer.load(s, A.to(DEV), B.to(DEV), alpha)
    return layer


@pytest.mark.parametrize("T,K,N", [(520, 512, 136), (1500, 1024, 520), (4096, 2048, 256)])
@pytest.mark.parametrize("fp8_base", [False, True])
def test_forward_right_behind_the_norm(T, K, N, fp8_base):
    from segmented_rank_gemm_gb300.norm import lora_rms_norm
    wl = workloads.synthetic(900 + T, T, K, N, S=4, ranks=[1, 16, 8, 3], R=16, base_frac=0.2)
    layer = _layer(wl, fp8_base)
    ids = wl.token_slot.to(DEV)
    rounds = 12
    xs = torch.randn(rounds, T, K, generator=torch.Generator().manual_seed(T)).to(BF16).to(DEV)
    w = torch.ones(K, dtype=BF16, device=DEV)
    n = torch.empty(T, K, dtype=BF16, device=DEV)
    xq = torch.empty(T, K, dtype=torch.float8_e4m3fn, device=DEV) if fp8_base else None
    sx = torch.empty(T, device=DEV) if fp8_base else None

    def run(i, y, pause):
        layer.set_batch(ids)
        pause()
        lora_rms_norm(xs[i], w, 1e-6, y=n, xq=xq, sx=sx)
        pause()
        if fp8_base:
            layer.forward_e4m3(n, xq, sx, y)
        else:
            layer.forward(n, y)
        pause()

    apart, behind = (torch.full((rounds, T, N), 9.0, dtype=BF16, device=DEV) for _ in range(2))
    for i in range(rounds):
        run(i, apart[i], torch.cuda.synchronize)
    for i in range(rounds):
        run(i, behind[i], lambda: None)
    torch.cuda.synchronize()
    assert layer.status() == 0
    assert torch.equal(apart, behind)
    if not fp8_base:
        wl.x = n.cpu()
        assert_parity(behind[-1], oracle_rows(wl), BF16, what="forward behind the norm")
    layer.close()
