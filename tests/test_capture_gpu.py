"""Every call between the projections, captured in one CUDA graph: a capture fails on a call that
allocates or synchronises, and a replay gives what the calls give one by one."""
import pytest
import torch

from segmented_rank_gemm_gb300 import workloads

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def test_every_call_in_one_graph():
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable
    from segmented_rank_gemm_gb300.lora import LoraLayer
    from segmented_rank_gemm_gb300.norm import lora_rms_norm
    B, page, hkv, G, D, T = 6, 16, 2, 4, 64, 640
    K, N = hkv * G * D, 256
    new = [1, 40, 0, 1, 500, 7]  # few rows a cache head and many
    wl = workloads.synthetic(71, T, K, N, S=4, ranks=[4, 8, 1, 8], R=8, base_frac=0.2)
    layer = LoraLayer(wl.W.to(DEV), wl.S, wl.R, T, fp8_base=True)
    for s, (A, Bm, alpha) in enumerate(wl.adapters):
        layer.load(s, A.to(DEV), Bm.to(DEV), alpha)
    g = torch.Generator().manual_seed(72)
    rand = lambda *s: torch.randn(*s, generator=g).to(BF16).to(DEV)  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    counts, ids = ints(new), ints([0, 3, -1, 1, 2, 2])
    first, last = ints([1] * B), ints([0, 1, 0, 0, 1, 0])
    k, v, q, w = rand(T, hkv, D), rand(T, hkv, D), rand(T, hkv * G, D), rand(K)
    pages, cache = PageTable(80, page, B, 40, T), KvCache(80, page, hkv, D, B)
    ko, vo, out = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
    h, n = rand(T, K), torch.empty(T, K, dtype=BF16, device=DEV)
    h0 = h.clone()
    xq = torch.empty(T, K, dtype=torch.float8_e4m3fn, device=DEV)
    sx, y = torch.empty(T, device=DEV), torch.empty(T, N, dtype=BF16, device=DEV)
    results = (pages.block_table, pages.kv_len, pages.q_offsets, pages.position, pages.kv_slot,
               pages.token_slot, pages.free_pages, pages.counts, ko, vo, out, h, n, xq.view(torch.uint8),
               sx, y)

    def step():
        pages.step(counts, ids)
        cache.append(k, v, pages.kv_slot)
        cache.read(pages.kv_slot, ko, vo)
        cache.attend(q, pages.q_offsets, pages.kv_len, pages.block_table, 500, out=out)
        lora_rms_norm(out.view(T, K), w, 1e-6, h, h, n, xq, sx)
        layer.set_batch(pages.token_slot)
        layer.forward_e4m3(n, xq, sx, y)
        pages.release(last)

    def reset():
        pages.release(first)
        pages.block_table.zero_()
        pages.free_pages.copy_(torch.arange(79, -1, -1))
        h.copy_(h0)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in results]
    reset()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (ko, vo, out, n, y):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results, want))
        assert pages.status()[3:] == (0, 0) and cache.status() == 0 and layer.status() == 0
        reset()
    layer.close()
    cache.close()
