"""Objects whose tensors are computed on the current stream are ready when they are there: a call on another
stream may be the first to read them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def test_a_rotary_is_ready_when_it_is_there():
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    cache, side = KvCache(4, 16, 1, 64, 2), torch.cuda.Stream()
    q, k = (torch.randn(40, h, 64, device=DEV).bfloat16() for h in (4, 1))
    at, slot = _ints(np.arange(40)), _ints(np.arange(40))
    want = cache.append_rotated(q, k, k, at, slot, Rotary(40, 64, theta=77.0))
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    rotary = Rotary(40, 64, theta=77.0)
    got = cache.append_rotated(q, k, k, at, slot, rotary, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    torch.cuda.synchronize()


def test_a_page_table_is_ready_when_it_is_there():
    from segmented_rank_gemm_gb300.kv import PageTable
    side, new = torch.cuda.Stream(), _ints([20, 3])
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    pages = PageTable(8, 16, 2, 4, 30)
    pages.step(new, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        assert pages.status() == (23, 5, 3, 0, 0) and pages.kv_len.tolist() == [20, 3]
        assert pages.kv_slot.tolist() == [*range(20), 32, 33, 34] + [-1] * 7
    torch.cuda.synchronize()
