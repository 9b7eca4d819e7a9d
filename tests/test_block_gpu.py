"""The attention half of a decoder block on the GPU: maps, norm, projections with an adapter a
row, cache and attention in one pass.  Each stage is compared with its 64-bit definition on the
rows that the pass itself handed to that stage, at the stage's own tolerance: projections as in
``gpu_helpers``, cached values exactly, attention at 2^-8 |o| + 2^-10 max|v| (the derivation is
test_kv_gpu's), norm rows at one rounding to bf16 and 2^-20.  Also lora_forward_e4m3, which takes
the norm's e4m3 rows.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from oracle import kv as ref
from segmented_rank_gemm_gb300 import workloads
from gpu_helpers import assert_parity

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def _np(t):
    return t.detach().float().cpu().numpy()


def _layer(wl, max_tokens, fp8_base):
    from segmented_rank_gemm_gb300.lora import LoraLayer
    layer = LoraLayer(wl.W.to(DEV), wl.S, wl.R, max_tokens, fp8_base=fp8_base)
    for s, ad in enumerate(wl.adapters):
        if ad is not None:
            layer.load(s, ad[0].to(DEV), ad[1].to(DEV), ad[2])
    return layer


def _e4m3_rows(x):
    xq, sx = fp8.quantize_rows(x)
    return (torch.from_numpy(xq).float().to(torch.float8_e4m3fn).to(DEV),
            torch.from_numpy(sx).to(DEV))


# ---------------------------------------------------------------------------------------
# lora_forward_e4m3
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,K,N", [(1, 64, 72), (3, 512, 320), (129, 256, 1040), (512, 1024, 264),
                                   (513, 256, 136), (1500, 512, 520)])
def test_given_rows_equal_the_layers_own(T, K, N):
    wl = workloads.synthetic(810 + T, T, K, N, S=6, ranks=[1, 16, 8, 3, 12, 2], R=16,
                             base_frac=0.15)
    layer = _layer(wl, T, True)
    x, ids = wl.x.to(DEV), wl.token_slot.to(DEV)
    own = layer(x, ids)
    launches = layer.launch_count()
    xq, sx = _e4m3_rows(_np(wl.x))
    layer.set_batch(ids)
    given = layer.forward_e4m3(x, xq, sx)
    torch.cuda.synchronize()
    assert torch.equal(given, own)
    assert layer.launch_count() == launches - 1  # no row quantiser
    # bytes are taken too, and the layer's own path still works after
    layer.set_batch(ids)
    assert torch.equal(layer.forward_e4m3(x, xq.view(torch.uint8), sx), own)
    assert torch.equal(layer(x, ids), own)
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("T", [40, 600])
def test_given_rows_feed_the_base_alone(T):
    # rows that are not x's: the base product takes them, the low-rank product takes x
    K, N = 256, 200
    wl = workloads.synthetic(830, T, K, N, S=4, ranks=8, R=8, base_frac=0.2)
    layer = _layer(wl, T, True)
    other = torch.randn(T, K, generator=torch.Generator().manual_seed(1)) * 3
    xq, sx = _e4m3_rows(_np(other))
    ids = wl.token_slot.to(DEV)
    layer.set_batch(ids)
    y = layer.forward_e4m3(wl.x.to(DEV), xq, sx)
    table = oracle.SlotTable(wl.adapters, K, N)
    delta = oracle.forward_rows(wl.x, torch.zeros(K, N, dtype=torch.float64), table, wl.token_slot)
    assert_parity(y, fp8.base_w8a8(_np(other), _np(wl.W)) + delta, BF16, what="given rows")
    layer.close()


def test_given_rows_refusals():
    from segmented_rank_gemm_gb300 import lora
    wl = workloads.synthetic(840, 20, 64, 64, S=2, ranks=4, R=4, base_frac=0.2)
    x, ids = wl.x.to(DEV), wl.token_slot.to(DEV)
    xq, sx = _e4m3_rows(_np(wl.x))
    y = torch.empty(20, 64, dtype=BF16, device=DEV)
    plain, layer = _layer(wl, 20, False), _layer(wl, 20, True)
    plain.set_batch(ids)
    with pytest.raises(lora.LoraError, match="e4m3 base"):
        plain.forward_e4m3(x, xq, sx)
    with pytest.raises(lora.LoraError) as e:
        layer.forward_e4m3(x, xq, sx)   # no batch yet
    assert e.value.code == lora.LORA_ESTATE
    layer.set_batch(ids)
    whole = torch.empty(20 * 64 + 64, dtype=torch.uint8, device=DEV)
    for bx, bq, bs, by in ((x, None, sx, y), (x, xq, None, y), (None, xq, sx, y), (x, xq, sx, None),
                           (x, whole[8:], sx, y), (x, y.view(torch.uint8).view(-1), sx, y),
                           (x, xq, y.view(torch.float32), y)):
        with pytest.raises(lora.LoraError) as e:
            lora.lora_forward_e4m3(layer.handle, bx, bq, bs, by, 20)
        assert e.value.code == lora.LORA_EINVAL
    with pytest.raises(lora.LoraError) as e:
        lora.lora_forward_e4m3(layer.handle, x, xq, sx, y, 19)
    assert e.value.code == lora.LORA_ESTATE
    for bad in (xq[:, :63], xq[:19], xq.float(), xq.cpu()):
        with pytest.raises(ValueError):
            layer.forward_e4m3(x, bad, sx)
    for bad in (sx[:19], sx.bfloat16(), sx.cpu()):
        with pytest.raises(ValueError):
            layer.forward_e4m3(x, xq, bad)
    layer.forward_e4m3(x, xq, sx, y)
    assert layer.status() == 0
    plain.close(), layer.close()


# ---------------------------------------------------------------------------------------
# the block
# ---------------------------------------------------------------------------------------

HQ, HKV, D, HIDDEN, S, PAGE, B = 8, 2, 64, 256, 5, 16, 6


class _Block:
    def __init__(self, fp8_base, max_tokens, rotate=None):
        from segmented_rank_gemm_gb300.block import AttentionBlock
        from segmented_rank_gemm_gb300.kv import KvCache, PageTable
        self.wl = [workloads.synthetic(850 + i, 1, K, N, S=S, ranks=[4, 8, 1, 8, 3], R=8)
                   for i, (K, N) in enumerate(((HIDDEN, HQ * D), (HIDDEN, HKV * D),
                                               (HIDDEN, HKV * D), (HQ * D, HIDDEN)))]
        self.layers = [_layer(wl, max_tokens, fp8_base) for wl in self.wl]
        g = torch.Generator().manual_seed(2)
        self.w = (1 + 0.2 * torch.randn(HIDDEN, generator=g)).bfloat16().to(DEV)
        self.cache = KvCache(200, PAGE, HKV, D, B)
        self.pages = PageTable(200, PAGE, B, 40, max_tokens)
        self.block = AttentionBlock(*self.layers, self.w, self.cache, rotate=rotate)
        self.fp8 = fp8_base
        self.kept = [([], []) for _ in range(B)]

    def check(self, i, rows, ids, got):
        """Projection i of the batch's rows against its definition."""
        wl, T = self.wl[i], len(ids)
        table = oracle.SlotTable(wl.adapters, wl.K, wl.N)
        if not self.fp8:
            want = oracle.forward_rows(rows.cpu(), wl.W, table, ids)
        else:
            if i < 3:
                b = self.block
                vals = _np(b.nq[:T]).astype(np.float64) * _np(b.sn[:T])[:, None]
                wq, sw = fp8.quantize_cols(_np(wl.W))
                base = (vals @ wq) * sw.astype(np.float64)
            else:
                base = fp8.base_w8a8(_np(rows), _np(wl.W))
            want = base + oracle.forward_rows(
                rows.cpu(), torch.zeros(wl.K, wl.N, dtype=torch.float64), table, ids)
        assert_parity(got, want, BF16, what="projection %d" % i)


def _rotate(q, k, position):
    # pairs (d, d + D / 2) turned by an angle that falls with d
    a = position[:, None, None].float() * 100.0 ** (-torch.arange(D // 2, device=DEV) / (D // 2))
    for t in (q, k):
        lo, hi = t[..., :D // 2].float(), t[..., D // 2:].float()
        t[..., :D // 2] = (lo * a.cos() - hi * a.sin()).to(t.dtype)
        t[..., D // 2:] = (lo * a.sin() + hi * a.cos()).to(t.dtype)


@pytest.mark.parametrize("fp8_base", [False, True])
def test_block_through_prompts_and_tokens(fp8_base):
    adapter = np.array([0, 3, -1, 1, 4, 2])
    blk = _Block(fp8_base, 700)
    g = torch.Generator().manual_seed(3)
    h64 = None
    for new in ([40, 3, 0, 130, 17, 1], [1, 1, 400, 1, 130, 1], [1] * 6, [1, 0, 1, 1, 1, 2]):
        T = sum(new)
        x, h = (torch.randn(T, HIDDEN, generator=g).bfloat16().to(DEV) for _ in range(2))
        h0 = h.clone()
        blk.pages.step(torch.tensor(new, dtype=torch.int32, device=DEV),
                       torch.tensor(adapter, dtype=torch.int32, device=DEV))
        y = blk.block.forward(x, h, blk.pages, max(new))
        torch.cuda.synchronize()
        assert blk.pages.status()[3] == 0 and blk.cache.status() == 0
        assert all(layer.status() == 0 for layer in blk.layers)
        ids = np.repeat(adapter, new).astype(np.int32)
        assert np.array_equal(blk.pages.token_slot[:T].cpu().numpy(), ids)
        b = blk.block
        assert torch.equal(h.cpu(), (x.float() + h0.float()).bfloat16().cpu())
        _, n64, _ = ref.rms_norm(_np(x), _np(h0), _np(blk.w), 1e-6)
        assert (np.abs(_np(b.n[:T]) - n64) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(n64)).all()
        q, k, v, ctx = (t[:T] for t in (b.qr, b.kr, b.vr, b.ctx))
        for i, got in enumerate((q, k, v)):
            blk.check(i, b.n[:T], torch.from_numpy(ids), got)
        q, k, v = (_np(t).reshape(T, -1, D) for t in (q, k, v))
        at, want = 0, []
        for r, c in enumerate(new):
            blk.kept[r][0].extend(ref.held(k[at:at + c]))
            blk.kept[r][1].extend(ref.held(v[at:at + c]))
            if c:
                want.append(ref.attend(q[at:at + c], np.array(blk.kept[r][0]),
                                       np.array(blk.kept[r][1]), D ** -0.5))
            at += c
        want = np.concatenate(want).reshape(T, -1)
        vmax = max(np.abs(np.array(kept[1])).max() for kept in blk.kept if kept[1])
        assert (np.abs(_np(ctx) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * vmax).all()
        blk.check(3, ctx, torch.from_numpy(ids), y)


@pytest.mark.parametrize("fp8_base", [False, True])
def test_block_in_a_graph(fp8_base):
    # single tokens of every request, captured with the page table's step; and the rotation
    # that is given runs between projections and cache
    eager, graph = (_Block(fp8_base, 64, _rotate) for _ in range(2))
    ones = torch.ones(B, dtype=torch.int32, device=DEV)
    ad = torch.tensor([0, 3, -1, 1, 4, 2], dtype=torch.int32, device=DEV)
    x, h = (torch.zeros(B, HIDDEN, dtype=BF16, device=DEV) for _ in range(2))
    y = torch.empty_like(x)
    g = torch.Generator().manual_seed(4)
    captured = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(captured):
        graph.pages.step(ones, ad)
        graph.block.forward(x, h, graph.pages, 1, y)
    for _ in range(20):
        xs, hs = (torch.randn(B, HIDDEN, generator=g).bfloat16().to(DEV) for _ in range(2))
        x.copy_(xs), h.copy_(hs)
        captured.replay()
        eager.pages.step(ones, ad)
        he = hs.clone()
        ye = eager.block.forward(xs, he, eager.pages, 1)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(h, he)
    assert eager.pages.kv_len.tolist() == graph.pages.kv_len.tolist() == [20] * B
    k = torch.ones(1, 1, D, dtype=BF16, device=DEV)
    _rotate(k, k.clone(), torch.tensor([5], device=DEV))
    assert not torch.equal(k, torch.ones_like(k))


def test_block_refusals():
    from segmented_rank_gemm_gb300.block import AttentionBlock
    blk = _Block(False, 16)
    q, k, v, o = blk.layers
    for bad in ((k, k, q, o), (q, k, v, k), (q, q, v, o), (o, k, v, o)):
        with pytest.raises(ValueError):
            AttentionBlock(*bad, blk.w, blk.cache)
    x = torch.zeros(17, HIDDEN, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        blk.block.forward(x, x.clone(), blk.pages, 1)
