"""The rotation, the shared prefixes, the encoder attention, the forks and the fused forwards: tensors of
another GPU, outputs that a call allocates on its own stream, calls of two caches and two layers at
the same time, and all of them in one captured graph."""
import pytest
import torch

from segmented_rank_gemm_gb300 import workloads

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_tensors_of_another_gpu_are_refused(monkeypatch):
    from segmented_rank_gemm_gb300 import kv
    from segmented_rank_gemm_gb300.lora import LORA_EINVAL, LoraError
    cache, pages = kv.KvCache(4, 16, 1, 64, 2), kv.PageTable(4, 16, 2, 2, 8)
    rotary = kv.Rotary(8, 64)
    k, q = torch.ones(2, 1, 64, dtype=BF16, device=DEV), torch.ones(2, 4, 64, dtype=BF16, device=DEV)
    table = ints(0, 1, 2, 3).view(2, 2)
    calls = [lambda: cache.append_rotated(q, k, k, ints(0, 1), ints(0, 1), rotary),
             lambda: cache.append_rotated(q, k, k, ints(0, 1), ints(0, 1), rotary, q_out=q.clone()),
             lambda: cache.attend(q, ints(0, 1, 2), ints(1, 1), table, 1, causal=False),
             lambda: cache.attend_shared(q, ints(0, 1, 2), ints(17, 17), table, 1, ints(0, 2), ints(0), ints(16),
                                         ints(16, 16)),
             lambda: pages.fork(ints(-1, -1)), lambda: pages.fork(ints(-1, -1), ints(0, 0)),
             lambda: pages.release(ints(0, 0))]
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
    assert cache.status() == 0
    cache.close()


def _layer(seed, K, N, T, **kw):
    from segmented_rank_gemm_gb300.lora import LoraLayer
    wl = workloads.synthetic(seed, T, K, N, S=4, ranks=[4, 8, 1, 8], R=8, base_frac=0.2)
    layer = LoraLayer(wl.W.to(DEV), wl.S, wl.R, T, **kw)
    for s, (A, B, alpha) in enumerate(wl.adapters):
        layer.load(s, A.to(DEV), B.to(DEV), alpha)
    return layer, wl


def _setup(seed, T=40, B=12, page=16, hkv=2, G=4, D=64):
    """A cache whose first request is a prompt that the others are forked from, and a batch."""
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable, Rotary
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g).to(BF16).to(DEV)  # noqa: E731
    cache, pages = KvCache(200, page, hkv, D, B), PageTable(200, page, B, 20, 150)
    rotary = Rotary(400, D)
    n = 100 + seed % 50
    pages.step(ints(n, *[0] * (B - 1)))
    cache.append_rotated(rand(n, hkv * G, D), rand(n, hkv, D), rand(n, hkv, D), pages.position[:n],
                         pages.kv_slot[:n], rotary)
    pages.fork(ints(-1, *[0] * (B - 1)))
    new = [0] + [1 + i % 6 for i in range(B - 1)]
    T = sum(new)
    pages.step(ints(*new))
    x = dict(q=rand(T, hkv * G, D), k=rand(T, hkv, D), v=rand(T, hkv, D))
    groups = (ints(1, B), ints(0), ints(n // page * page))
    torch.cuda.synchronize()

    def run(stream=None, out=None, q_out=None, workspace=None):
        q = cache.append_rotated(x["q"], x["k"], x["v"], pages.position[:T], pages.kv_slot[:T], rotary,
                                 q_out=q_out, stream=stream)
        args = (q, pages.q_offsets, pages.kv_len, pages.block_table, 6)
        a = cache.attend_shared(*args, *groups, pages.shared_len, stream=stream, out=out, workspace=workspace)
        return a, cache.attend(*args, stream=stream, causal=False)

    return cache, run, x["q"]


def test_outputs_on_a_stream_are_its_memory():
    # the default stream is busy with memory that the calls' outputs must not be
    cache, run, _ = _setup(3)
    layer, wl = _layer(5, 256, 512, 64)
    x, ids = wl.x.to(DEV), wl.token_slot.to(DEV)
    want = [t.clone() for t in run()]
    layer.set_batch(ids)
    want.append(layer.forward_fused(x, activation="silu").clone())
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        junk = [torch.empty(1 << 16, dtype=torch.uint8, device=DEV).fill_(7) for _ in range(8)]
        del junk
        torch.cuda._sleep(2_000_000)
        layer.set_batch(ids, stream)
        got = [*run(stream), layer.forward_fused(x, activation="silu", stream=stream)]
        more = [torch.empty(1 << 16, dtype=torch.uint8, device=DEV).fill_(9) for _ in range(8)]
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del more
    torch.cuda.synchronize()
    layer.close()
    cache.close()


def test_two_at_a_time():
    # caches and layers of their own, on streams of their own, give what they give one by one
    parts = []
    for seed in (11, 12):
        cache, run, _ = _setup(seed)
        small, wl = _layer(20 + seed, 256, 1024, 300)
        large, wl2 = _layer(30 + seed, 256, 1032, 700, fp8_base=seed == 12)
        parts.append((cache, run, [(small, wl.x.to(DEV), wl.token_slot.to(DEV)),
                                   (large, wl2.x.to(DEV), wl2.token_slot.to(DEV))], torch.cuda.Stream()))

    def go(part, stream):
        out = list(part[1](stream))
        for layer, x, ids in part[2]:
            layer.set_batch(ids, stream)
            u = layer.forward_fused(x, stream=stream)
            out.append(layer.forward_fused(x, activation="gelu", factor=u, residual=u, stream=stream))
        return out

    want = []
    for part in parts:
        want.append([t.clone() for t in go(part, part[3])])
        torch.cuda.synchronize()
    for _ in range(30):
        got = [go(part, part[3]) for part in parts]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    for cache, _, layers, _ in parts:
        assert cache.status() == 0 and all(layer.status() == 0 for layer, _, _ in layers)


def test_every_call_in_one_graph():
    cache, run, q = _setup(21)
    layer, wl = _layer(41, 256, 264, 90)
    x, ids = wl.x.to(DEV), wl.token_slot.to(DEV)
    T = q.shape[0]
    out, q_out, ws = torch.empty_like(q), torch.empty_like(q), cache.shared_workspace(T, 8)
    y, f = torch.empty(90, 264, dtype=BF16, device=DEV), torch.ones(90, 264, dtype=BF16, device=DEV)
    results = [out, q_out, y]

    def step():
        run(out=out, q_out=q_out, workspace=ws)
        layer.set_batch(ids)
        layer.forward_fused(x, y, bias=f[0], activation="gelu_tanh", factor=f, residual=f)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in results]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in results:
            t.fill_(3.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results, want))
    assert cache.status() == 0 and layer.status() == 0
