"""Tensors of another GPU than the current one are refused before anything is launched.  (One GPU is
enough: the current device is named another one's number for the binding.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def test_tensors_of_another_gpu_are_refused(monkeypatch):
    from segmented_rank_gemm_gb300 import kv
    from segmented_rank_gemm_gb300.lora import LORA_EINVAL, LoraError
    from segmented_rank_gemm_gb300.norm import lora_rms_norm, rms_norm
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cache = kv.KvCache(4, 16, 1, 64, 2)
    pages = kv.PageTable(4, 16, 2, 2, 8)
    k, q = torch.ones(2, 1, 64, dtype=BF16, device=DEV), torch.ones(2, 4, 64, dtype=BF16, device=DEV)
    x, w = torch.ones(3, 64, dtype=BF16, device=DEV), torch.ones(64, dtype=BF16, device=DEV)
    y, h = torch.empty_like(x), torch.empty_like(x)
    xq, sx = torch.empty(3, 64, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(3, device=DEV)
    calls = [lambda: cache.append(k, k, ints(0, 1)), lambda: cache.read(ints(0, 1)),
             lambda: cache.read(ints(0, 1), k.clone(), k.clone()),
             lambda: cache.attend(q, ints(0, 1, 2), ints(1, 1), ints(0, 1).view(2, 1), 1),
             lambda: pages.step(ints(1, 1)), lambda: pages.step(ints(1, 1), ints(0, 1)),
             lambda: pages.release(ints(1, 1)), lambda: rms_norm(x, w),
             lambda: lora_rms_norm(x, w, 1e-6, x.clone(), h, y, xq, sx)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        for call in calls:
            with pytest.raises(LoraError) as e:
                call()
            assert e.value.code == LORA_EINVAL
    for call in calls:
        call()
    torch.cuda.synchronize()
    assert cache.status() == 0
    cache.close()
