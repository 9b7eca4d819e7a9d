"""The attention block on a stream that is not the current one, and what it refuses before it has
changed anything."""
import numpy as np
import pytest
import torch

from test_block_gpu import B, HIDDEN, _Block, _rotate

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def _batch(blk, new, seed):
    g = torch.Generator().manual_seed(seed)
    x, h = (torch.randn(sum(new), HIDDEN, generator=g).to(BF16).to(DEV) for _ in range(2))
    ids = torch.tensor([0, 3, -1, 1, 4, 2], dtype=torch.int32, device=DEV)
    return torch.tensor(new, dtype=torch.int32, device=DEV), ids, x, h


@pytest.mark.parametrize("handle", [False, True])
def test_rotation_on_the_blocks_stream(handle):
    seen = []

    def rotate(q, k, position):
        seen.append(torch.cuda.current_stream().cuda_stream)
        _rotate(q, k, position)

    here, there = (_Block(False, 200, rotate) for _ in range(2))
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    for i, new in enumerate(([40, 3, 0, 100, 17, 1], [1, 1, 60, 1, 100, 1], [1] * 6)):
        counts, ids, x, h = _batch(here, new, i)
        h2, y2 = h.clone(), torch.empty_like(x)
        here.pages.step(counts, ids)
        y = here.block.forward(x, h, here.pages, max(new))
        torch.cuda.synchronize()
        assert seen.pop() == torch.cuda.current_stream().cuda_stream
        # the current stream is busy while the block runs beside it
        torch.cuda._sleep(20_000_000)
        there.pages.step(counts, ids, given)
        there.block.forward(x, h2, there.pages, max(new), y2, given)
        side.synchronize()
        assert seen.pop() == side.cuda_stream and not seen
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(h, h2)
        assert there.cache.status() == 0 and there.pages.status()[3] == 0
    # the default stream, by its handle
    here.pages.step(counts, ids, 0)
    here.block.forward(x, h, here.pages, 1, stream=0)
    assert seen.pop() == torch.cuda.default_stream().cuda_stream
    torch.cuda.synchronize()


def test_refusals_come_before_the_residual_changes():
    from segmented_rank_gemm_gb300.block import AttentionBlock
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable
    blk = _Block(False, 60)
    new = [3, 1, 1, 20, 1, 1]
    counts, ids, x, h = _batch(blk, new, 7)
    before = h.clone()
    small = PageTable(200, 16, B, 40, sum(new) - 1)
    pages = PageTable(200, 32, B, 40, 60)
    more = PageTable(200, 16, B + 1, 40, 60)
    for table, max_q in ((small, 20), (pages, 20), (more, 20), (blk.pages, 0), (blk.pages, -3)):
        with pytest.raises(ValueError):
            blk.block.forward(x, h, table, max_q)
        assert torch.equal(h, before)
    slots = torch.arange(200 * 16, dtype=torch.int32, device=DEV)
    k, v = blk.cache.read(slots)
    assert not k.any() and not v.any()
    # heads that the cache's do not divide
    q, kl, vl, o = blk.layers
    with pytest.raises(ValueError):
        AttentionBlock(q, kl, vl, o, blk.w, KvCache(8, 16, 3, 64, B))


def _wrong_outputs(T, N):
    return (torch.empty(T - 1, N, dtype=BF16, device=DEV), torch.empty(T, N - 8, dtype=BF16, device=DEV),
            torch.empty(T, N, device=DEV), torch.empty(T, N, dtype=BF16),
            torch.empty(T, N + 8, dtype=BF16, device=DEV)[:, :N])


def test_outputs_that_do_not_fit_are_refused():
    from segmented_rank_gemm_gb300 import workloads
    from test_block_gpu import _layer
    blk = _Block(False, 60)
    new = [3, 1, 1, 20, 1, 1]
    counts, ids, x, h = _batch(blk, new, 7)
    before = h.clone()
    blk.pages.step(counts, ids)
    for y in _wrong_outputs(27, HIDDEN):
        with pytest.raises(ValueError):
            blk.block.forward(x, h, blk.pages, 20, y)
        assert torch.equal(h, before)
    for fp8_base in (False, True):
        wl = workloads.synthetic(5, 40, 64, 72, S=2, ranks=4, R=4, base_frac=0.2)
        layer = _layer(wl, 40, fp8_base)
        xl = wl.x.to(DEV)
        layer.set_batch(wl.token_slot.to(DEV))
        xq = torch.zeros(40, 64, dtype=torch.uint8, device=DEV)
        sx = torch.ones(40, device=DEV)
        for y in _wrong_outputs(40, 72):
            with pytest.raises(ValueError):
                layer.forward(xl, y)
            if fp8_base:
                with pytest.raises(ValueError):
                    layer.forward_e4m3(xl, xq, sx, y)
        assert layer.status() == 0
        layer.close()


def test_layers_that_do_not_fit_are_refused():
    from segmented_rank_gemm_gb300.block import AttentionBlock
    from segmented_rank_gemm_gb300.lora import LoraLayer
    blk = _Block(False, 16)
    q, k, v, o = blk.layers
    wide = LoraLayer(torch.zeros(q.N, HIDDEN + 8, dtype=BF16, device=DEV), 5, 8, 16)
    f32 = [LoraLayer(torch.zeros(layer.K, layer.N, device=DEV), 5, 8, 16) for layer in blk.layers]
    for bad in ((q, k, v, wide), (f32[0], k, v, o), (q, f32[1], v, o), (q, k, f32[2], o), (q, k, v, f32[3]),
                f32):
        with pytest.raises(ValueError):
            AttentionBlock(*bad, blk.w, blk.cache)


@pytest.mark.parametrize("fp8_base", [False, True])
def test_batch_without_rows(fp8_base):
    blk = _Block(fp8_base, 60, _rotate)
    counts, ids, x, h = _batch(blk, [2, 0, 0, 3, 0, 0], 8)
    blk.pages.step(counts, ids)
    blk.block.forward(x, h, blk.pages, 3)
    blk.pages.step(torch.zeros_like(counts), ids)
    y = blk.block.forward(x[:0], h[:0], blk.pages, 1)
    assert y.shape == (0, HIDDEN) and y.dtype == BF16
    torch.cuda.synchronize()
    assert blk.pages.kv_len.tolist() == [2, 0, 0, 3, 0, 0] and blk.cache.status() == 0
    assert all(layer.status() == 0 for layer in blk.layers)
