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


@pytest.mark.parametrize("scale,size", [(0.0, 1e33), (-0.0, 1.0), (3e-33, 1e32), (-2e-31, 1e30),
                                        (1e-36, 3e36), (1e-30, 1.0), (2e-38, 1e5)])
@pytest.mark.parametrize("D", [64, 128])
def test_tiny_scales_on_both_sides_of_the_row_threshold(scale, size, D):
    # queries so large that scores are of ordinary size, or vanish; 24 rows a cache head and less go to
    # one kernel, 28 and more to the other
    kv, new = [130, 77, 300, 65, 40], [1, 6, 7, 40, 2]
    s = Setup(kv, D, 1, 64, seed=42)
    q = s.queries(new, 4, spread=size)
    out = s.attend(q.to(DEV), new, scale)
    assert s.cache.status() == 0
    _close(out, s.expected(q, new, scale), np.abs(s.hv).max())


@pytest.mark.parametrize("g", [4.8e37, 4.9e37, 1e38, 3e38])
def test_largest_scales_of_the_cache(g):
    # the scale of a group is max|x| / (7 g) in fp32: refused where 7 g is none
    from segmented_rank_gemm_gb300.kv import KvCache
    from segmented_rank_gemm_gb300.lora import LORA_EINVAL, LoraError
    if not np.isfinite(np.float32(7) * np.float32(g)):
        for scales in ((g, 1.0), (1.0, g)):
            with pytest.raises(LoraError) as e:
                KvCache(4, 16, 2, 64, 1, *scales)
            assert e.value.code == LORA_EINVAL
        return
    gen = torch.Generator().manual_seed(43)
    k, v = ((torch.rand(64, 2, 64, generator=gen) * 2 - 1).mul(3e38).bfloat16() for _ in range(2))
    cache = KvCache(4, 16, 2, 64, 1, g, g)
    slots = _ints(np.arange(64))
    cache.append(k.to(DEV), v.to(DEV), slots)
    for got, x in zip(cache.read(slots), (k, v)):
        want = torch.from_numpy(ref.held(_np(x), g).astype(np.float32)).bfloat16()
        assert want.abs().max() > 1e38 and torch.equal(got.cpu(), want)
    cache.close()
