"""The scales of the cache and of the attention at the ends of their ranges."""
import numpy as np
import pytest
import torch

from oracle import kv as ref
from test_kv_gpu import Setup, _close, _ints, _np

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("scale,k_scale,fits", [
    (1e30, 1e30, False), (-1e30, 1e30, False), (3e38, 1.0, False), (1e37, 1.0, False),
    (1e30, 1e6, True), (-1e36, 1.0, True), (3e38, 1e-6, True)])
def test_products_of_scales_that_overflow_are_refused(scale, k_scale, fits):
    from segmented_rank_gemm_gb300.lora import LORA_EINVAL, LoraError
    kv, new = [20, 70], [1, 30]  # few rows a cache head, many
    s = Setup(kv, 64, 1, 16, seed=41, k_scale=k_scale, spread=k_scale)
    q = torch.zeros(31, 4, 64, dtype=torch.bfloat16)
    out = torch.full_like(q, 7.0, device=DEV)
    if fits:
        s.attend(q.to(DEV), new, scale, out=out)
        _close(out, s.expected(q, new, scale), np.abs(s.hv).max())
    else:
        with pytest.raises(LoraError) as e:
            s.attend(q.to(DEV), new, scale, out=out)
        assert e.value.code == LORA_EINVAL and (out == 7).all()
    assert s.cache.status() == 0
