"""Outputs that the calls allocate themselves, on a stream that is not the current one: memory that
the current stream still has work for is not written on the other."""
import pytest
import torch

from segmented_rank_gemm_gb300 import workloads

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def _cases():
    """(name, the call with stream=, bytes of its output)"""
    from segmented_rank_gemm_gb300.kv import KvCache
    from segmented_rank_gemm_gb300.lora import LoraLayer, on_stream
    from segmented_rank_gemm_gb300.norm import rms_norm
    from test_block_gpu import HIDDEN, B, _Block
    g = torch.Generator().manual_seed(3)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    T, hkv, D = 2048, 2, 128
    cache = KvCache(T // 16, 16, hkv, D, 1)
    k, v = (torch.randn(T, hkv, D, generator=g).to(BF16).to(DEV) for _ in range(2))
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    cache.append(k, v, slots)
    yield "read", lambda stream: cache.read(slots, stream=stream), T * hkv * D * 2
    q = torch.randn(512, 8, D, generator=g).to(BF16).to(DEV)
    off, lens, table = ints([0, 512]), ints([T]), slots[:T // 16].view(1, -1)
    yield "attend", lambda stream: cache.attend(q, off, lens, table, 512, stream=stream), q.numel() * 2
    x = torch.randn(1024, 1024, generator=g).to(BF16).to(DEV)
    w = torch.ones(1024, dtype=BF16, device=DEV)
    yield "norm", lambda stream: rms_norm(x, w, stream=stream), x.numel() * 2
    for fp8 in (False, True):
        wl = workloads.synthetic(5, 600, 256, 1024, S=2, ranks=8, R=8, base_frac=0.2)
        layer = LoraLayer(wl.W.to(DEV), wl.S, wl.R, wl.T, fp8_base=fp8)
        for s, (A, Bm, alpha) in enumerate(wl.adapters):
            layer.load(s, A.to(DEV), Bm.to(DEV), alpha)
        xl, ids = wl.x.to(DEV), wl.token_slot.to(DEV)
        if not fp8:
            yield "forward", lambda stream: layer(xl, ids, stream=stream), 600 * 1024 * 2
            continue
        xq = torch.zeros(600, 256, dtype=torch.float8_e4m3fn, device=DEV)
        xq.copy_(torch.randn(600, 256, generator=g).to(DEV))
        sx = torch.rand(600, generator=g).to(DEV)

        def given(stream):
            layer.set_batch(ids, stream)
            return layer.forward_e4m3(xl, xq, sx, stream=stream)
        yield "forward_e4m3", given, 600 * 1024 * 2
    blk = _Block(False, 30 * B)
    thirty, none, all_of_them = ints([30] * B), ints([0] * B), ints([1] * B)
    xb = torch.randn(30 * B, HIDDEN, generator=g).to(BF16).to(DEV)
    hb = torch.zeros_like(xb)

    def block(stream):
        blk.pages.step(thirty, none, stream)
        y = blk.block.forward(xb, hb, blk.pages, 30, stream=stream)
        blk.pages.release(all_of_them, stream)
        with on_stream(stream):
            hb.zero_()
        return y
    yield "block", block, xb.numel() * 2


def _flat(x):
    return x if isinstance(x, torch.Tensor) else torch.cat(x)


def test_memory_is_the_calls_streams():
    side = torch.cuda.Stream()
    for name, call, size in _cases():
        want = _flat(call(None)).clone()
        torch.cuda.synchronize()
        for given in (side, side.cuda_stream):
            # memory of the output's size, free again, which the current stream has yet to write
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            pending = torch.empty(size, dtype=torch.uint8, device=DEV)
            torch.cuda._sleep(100_000_000)
            pending.fill_(0x77)
            del pending
            got = call(given)
            side.synchronize()
            torch.cuda.synchronize()
            assert torch.equal(_flat(got), want), name
            del got
