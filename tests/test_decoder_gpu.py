"""Both halves of a decoder block over the operators between and in its projections: rotation on the
way into the cache, prefixes shared by forked requests, gate times up and the residual in the
products' epilogues -- against the calls one by one, which their own tests hold to 64 bits, and the
MLP's rows against the oracle's sums of the rows that the GPU gave it.

Tolerance of the MLP: as in the fused products' tests, 2^-8 of the result for its rounding, 2e-3 for a
sum's error, passed by SiLU (slope at most 1.1) and multiplied by the factor.
"""
import numpy as np
import pytest
import torch

import oracle
from segmented_rank_gemm_gb300 import workloads

pytestmark = pytest.mark.gpu

DEV = "cuda"
HIDDEN, HEADS, KV, D, WIDTH = 256, 8, 2, 64, 512


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _layer(seed, K, N, T, e4m3=False):
    from segmented_rank_gemm_gb300.lora import LoraLayer
    wl = workloads.synthetic(seed, 1, K, N, S=3, ranks=[8, 4, 16], R=16, w_std=0.06)
    layer = LoraLayer(wl.W.to(DEV), 3, 16, T, fp8_base=e4m3)
    for s, (A, B, alpha) in enumerate(wl.adapters):
        layer.load(s, A.to(DEV), B.to(DEV), alpha)
    return layer, wl


def _attention(T, cache, e4m3=False, **kw):
    from segmented_rank_gemm_gb300.block import AttentionBlock
    layers = [_layer(30 + i, K, N, T, e4m3 and i < 3)[0] for i, (K, N) in enumerate(
        ((HIDDEN, HEADS * D), (HIDDEN, KV * D), (HIDDEN, KV * D), (HEADS * D, HIDDEN)))]
    w = (1 + 0.1 * torch.randn(HIDDEN, generator=torch.Generator().manual_seed(9))).bfloat16().to(DEV)
    return AttentionBlock(*layers, w, cache, **kw)


def _mlp(T, e4m3=False):
    from segmented_rank_gemm_gb300.block import MlpBlock
    made = [_layer(40 + i, K, N, T, e4m3 and i < 2) for i, (K, N) in enumerate(
        ((HIDDEN, WIDTH), (HIDDEN, WIDTH), (WIDTH, HIDDEN)))]
    w = torch.ones(HIDDEN, dtype=torch.bfloat16, device=DEV)
    return MlpBlock(*[m[0] for m in made], w), [m[1] for m in made]


def _rows(T, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, HIDDEN, generator=g) * scale).bfloat16().to(DEV)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_attention_block_is_its_calls(e4m3, interleaved):
    """A prompt, forked into samples, which then go on: forward, and the same calls one by one."""
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable, Rotary
    from segmented_rank_gemm_gb300.norm import lora_rms_norm
    T, B, page = 160, 6, 16
    rotary = Rotary(400, 32, interleaved=interleaved)
    caches = [KvCache(80, page, KV, D, B) for _ in range(2)]
    tables = [PageTable(80, page, B, 12, T) for _ in range(2)]
    block = _attention(T, caches[0], e4m3, rotary=rotary, share=True)
    other = _attention(T, caches[1], e4m3, rotary=rotary, share=True)
    groups = (_ints([1, B]), _ints([0]), _ints([112]))
    for step, (new, fork) in enumerate((([120, 0, 0, 0, 0, 0], False), ([0, 9, 9, 1, 30, 2], True),
                                        ([1, 1, 1, 1, 1, 0], True), ([0, 1, 2, 3, 1, 1], True))):
        n = sum(new)
        ids = _ints([0, 1, -1, 2, 1, 0])
        if step == 1:
            for t in tables:
                t.fork(_ints([-1] + [0] * (B - 1)))
        for t in tables:
            t.step(_ints(new), ids)
        x, h = _rows(n, step), _rows(n, 90 + step, 3.0)
        h2 = h.clone()
        y = block.forward(x, h, tables[0], max(new), groups=groups if fork else None)
        # the same calls
        t, c = tables[1], caches[1]
        rows, nq, sn = other.n[:n], None, None
        if e4m3:
            nq, sn = other.nq[:n], other.sn[:n]
        lora_rms_norm(x, other.norm_weight, other.eps, h2, h2, rows, nq, sn)
        out = []
        for layer in (other.q, other.k, other.v):
            layer.set_batch(t.token_slot[:n])
            out.append(layer.forward_e4m3(rows, nq, sn) if e4m3 else layer.forward(rows))
        q, k, v = out[0].view(n, HEADS, D), out[1].view(n, KV, D), out[2].view(n, KV, D)
        q = c.append_rotated(q, k, v, t.position[:n], t.kv_slot[:n], rotary)
        if fork:
            ctx = c.attend_shared(q, t.q_offsets, t.kv_len, t.block_table, max(new), *groups, t.shared_len)
        else:
            ctx = c.attend(q, t.q_offsets, t.kv_len, t.block_table, max(new))
        other.o.set_batch(t.token_slot[:n])
        want = other.o.forward(ctx.view(n, HEADS * D))
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(block.ctx[:n], ctx.view(n, HEADS * D))
        assert torch.equal(y, want) and y.abs().sum() > 0
        # without sharing: the same sums in another order
        alone = c.attend(q, t.q_offsets, t.kv_len, t.block_table, max(new))
        assert (alone.float() - ctx.float()).abs().max() <= 2.0 ** -7 * 4
        for t, c in zip(tables, caches):
            assert c.status() == 0 and t.status()[3] == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 70, 600])
def test_mlp_block_against_the_oracle(T, e4m3):
    from oracle import fp8
    mlp, wls = _mlp(T, e4m3)
    ids = torch.from_numpy(np.random.default_rng(T).integers(-1, 3, T).astype(np.int32))
    for residual in (False, True):
        x, h = _rows(T, 5), _rows(T, 6, 2.0)
        hsum = (x.float() + h.float()).bfloat16()
        y = mlp.forward(x, h, ids.to(DEV), residual=residual)
        torch.cuda.synchronize()
        assert torch.equal(h, hsum)
        n, mid = mlp.n[:T].clone(), mlp.mid[:T].clone()
        mlp.up.set_batch(ids.to(DEV))
        given = dict(xq=mlp.nq[:T], sx=mlp.sn[:T]) if e4m3 else {}
        up = mlp.up.forward_fused(n, **given)
        torch.cuda.synchronize()

        def sums(wl, rows, quantised):
            table, K, N = oracle.SlotTable(wl.adapters, wl.K, wl.N), wl.K, wl.N
            if not quantised:
                return oracle.forward_rows(rows.cpu(), wl.W, table, ids)
            delta = oracle.forward_rows(rows.cpu(), torch.zeros(K, N, dtype=torch.float64), table, ids)
            xq = mlp.nq[:T].float().cpu().double().numpy() * mlp.sn[:T].cpu().double().numpy()[:, None]
            wq, sw = fp8.quantize_cols(wl.W.float().numpy())
            return xq @ wq * sw.astype(np.float64) + delta

        v, u = sums(wls[0], n, e4m3), up.cpu().double().numpy()
        want = v / (1 + np.exp(-v)) * u
        lim = 2.0 ** -8 * np.abs(want) + 1.1 * 2e-3 * np.abs(u) + 2.0 ** -18 * np.abs(want)
        assert (np.abs(mid.cpu().double().numpy() - want) <= lim).all()
        want = sums(wls[2], mid, False) + (h.cpu().double().numpy() if residual else 0)
        lim = 2.0 ** -8 * np.abs(want) + 2e-3 + (2.0 ** -18 * np.abs(want) if residual else 0)
        assert (np.abs(y.cpu().double().numpy() - want) <= lim).all()
    for layer in (mlp.gate, mlp.up, mlp.down):
        assert layer.status() == 0


def test_a_block_in_a_graph_on_a_stream_and_in_place():
    """Attention and MLP, rotation and shared prefixes, captured with the step that maps them."""
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable, Rotary
    T, B, page = 64, 9, 16
    cache, pages, rotary = KvCache(90, page, KV, D, B), PageTable(90, page, B, 10, T), Rotary(200, 64)
    block, (mlp, _) = _attention(T, cache, rotary=rotary, share=True), _mlp(T)
    pages.step(_ints([40] + [0] * 8), _ints([1] * B))
    x, h = _rows(40, 1), _rows(40, 2)
    block.forward(x, h, pages, 40)
    pages.fork(_ints([-1] + [0] * 8))
    torch.cuda.synchronize()
    state = {k: getattr(pages, k).clone() for k in ("kv_len", "block_table", "counts", "shared_len")}
    groups = (_ints([1, B]), _ints([0]), _ints([32]))
    new, ids = _ints([0] + [2] * 8), _ints([1] * B)
    x, h, y = _rows(16, 3), _rows(16, 4), torch.empty(16, HIDDEN, dtype=torch.bfloat16, device=DEV)
    h0 = h.clone()

    def step(stream=None):
        pages.step(new, ids, stream)
        block.forward(x, h, pages, 2, y=y, stream=stream, groups=groups)
        mlp.forward(y, h, pages.token_slot, y=h, residual=True, stream=stream)

    def reset():
        torch.cuda.synchronize()
        for k, v in state.items():
            getattr(pages, k).copy_(v)
        h.copy_(h0)
        torch.cuda.synchronize()

    step()
    torch.cuda.synchronize()
    want = h.clone()
    assert torch.isfinite(want.float()).all() and not torch.equal(want, h0)
    reset()
    stream = torch.cuda.Stream()
    step(stream)
    stream.synchronize()
    assert torch.equal(h, want)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want)
    assert cache.status() == 0 and pages.status()[3] == 0


def test_blocks_refuse_what_does_not_fit():
    from segmented_rank_gemm_gb300.block import MlpBlock
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable, Rotary
    cache, pages = KvCache(8, 16, KV, D, 2), PageTable(8, 16, 2, 4, 8)
    with pytest.raises(ValueError):
        _attention(8, cache, rotary=Rotary(4, 32), rotate=lambda q, k, p: None)
    with pytest.raises(ValueError):
        _attention(8, cache, rotary=Rotary(4, 128))
    block = _attention(8, cache)
    pages.step(_ints([2, 1]))
    with pytest.raises(ValueError):  # made without share
        block.forward(_rows(3, 1), _rows(3, 2), pages, 2, groups=(_ints([0, 2]), _ints([0]), _ints([0])))
    mlp, _ = _mlp(8)
    ids = _ints([0] * 8)
    w = mlp.norm_weight
    for args in ((mlp.gate, mlp.down, mlp.up, w), (mlp.gate, mlp.up, block.q, w), (mlp.gate, mlp.up, mlp.down, w, "tanh"),
                 (mlp.gate, _layer(1, HIDDEN, WIDTH, 8, True)[0], mlp.down, w)):
        with pytest.raises(ValueError):
            MlpBlock(*args)
    x, h = _rows(8, 1), _rows(8, 2)
    for change in (dict(x=_rows(9, 1), h=_rows(9, 2)), dict(token_slot=ids[:5]), dict(y=x.float()), dict(y=x[:4])):
        before = h.clone()
        with pytest.raises(ValueError):
            mlp.forward(**{**dict(x=x, h=h, token_slot=ids), **change})
        assert torch.equal(h, before)
    assert mlp.forward(x[:0], h[:0], ids).shape == (0, HIDDEN)
    mlp.forward(x, h, ids)
