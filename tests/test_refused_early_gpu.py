"""What a block's pass refuses, it refuses before the running residual and the cache change: a caller
mends the argument and calls again."""
import pytest
import torch

from test_decoder_gpu import D, HIDDEN, KV, _attention, _ints, _mlp, _rows

pytestmark = pytest.mark.gpu

BF16, DEV = torch.bfloat16, "cuda"


def _across(h):
    """A dense output that shares some of h's memory (h's rows are in the middle of a larger array)."""
    base = h._base
    return base[1:1 + h.shape[0]]


def _in_the_middle(T, seed):
    h = torch.empty(T + 8, HIDDEN, dtype=BF16, device=DEV)[4:4 + T]
    return h.copy_(_rows(T, seed))


@pytest.mark.parametrize("residual", [False, True])
def test_mlp_block(residual):
    from segmented_rank_gemm_gb300.lora import LoraError
    mlp, _ = _mlp(8)
    x, h, ids = _rows(8, 1), _in_the_middle(8, 2), _ints([0, 1, -1, 2, 0, 0, 1, 1])
    before = h.clone()
    odd = torch.empty(8 * HIDDEN + 8, dtype=BF16, device=DEV)[4:4 + 8 * HIDDEN].view(8, HIDDEN)
    bad = [dict(token_slot=ids.long()), dict(token_slot=ids.cpu()), dict(token_slot=ids.float()),
           dict(token_slot=ids.repeat(2)[::2]), dict(token_slot=ids.view(4, 2)),
           dict(y=_across(h)), dict(y=odd), dict(y=x.cpu())]
    if not residual:
        bad.append(dict(y=h))  # the residual would be lost
    else:  # rows that the products' epilogue does not take
        wide = torch.empty(8, HIDDEN + 4, dtype=BF16, device=DEV)
        bad += [dict(h=wide[:, :HIDDEN].copy_(h)), dict(h=odd.clone().view(-1)[:0]),
                dict(h=torch.empty(8 * HIDDEN + 8, dtype=BF16, device=DEV)[4:4 + 8 * HIDDEN].view(8, HIDDEN).copy_(h))]
    for change in bad:
        args = {**dict(x=x, h=h, token_slot=ids), **change}
        kept = args["h"].clone()
        with pytest.raises((ValueError, LoraError)):
            mlp.forward(**args, residual=residual)
        torch.cuda.synchronize()
        assert torch.equal(args["h"], kept) and torch.equal(h, before), list(change)
    # after what was mended: as if nothing had been tried
    y = mlp.forward(x, h, ids, residual=residual)
    other = before.clone()
    want = mlp.forward(x, other, ids, residual=residual)
    torch.cuda.synchronize()
    assert torch.equal(h, other) and torch.equal(y, want)


def test_mlp_block_takes_strided_residual_rows():
    mlp, _ = _mlp(8)
    x, ids = _rows(8, 1), _ints([0, 1, -1, 2, 0, 0, 1, 1])
    wide = torch.zeros(8, HIDDEN + 8, dtype=BF16, device=DEV)
    h, dense = wide[:, :HIDDEN], _rows(8, 2)
    h.copy_(dense)
    y = mlp.forward(x, h, ids, residual=True)
    want = mlp.forward(x, dense, ids, residual=True)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(h, dense) and not wide[:, HIDDEN:].any()


def test_attention_block():
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable, Rotary
    from segmented_rank_gemm_gb300.lora import LoraError
    B, page = 3, 16
    cache, pages = KvCache(12, page, KV, D, B), PageTable(12, page, B, 4, 8)
    block = _attention(8, cache, share=True, rotary=Rotary(64, D))
    pages.step(_ints([4, 2, 1]))
    x, h = _rows(7, 1), _in_the_middle(7, 2)
    before = h.clone()
    good = (_ints([0, 2]), _ints([0]), _ints([0]))
    odd = torch.empty(7 * HIDDEN + 8, dtype=BF16, device=DEV)[4:4 + 7 * HIDDEN].view(7, HIDDEN)
    bad = [dict(groups=(g.long(), r, n)) for g, r, n in (good,)]
    bad += [dict(groups=g) for g in (
        (good[0].cpu(), *good[1:]), (good[0], good[1].long(), good[2]), (good[0], good[1], good[2].cpu()),
        (_ints([0]), *good[1:]), (_ints([0, 1, 2, 3, 3]), _ints([0] * 4), _ints([0] * 4)),
        (_ints([0, 1, 2]), *good[1:]), (good[0], good[1], good[2][:0]),
        (_ints([0, 0, 2, 0])[::2], *good[1:]), good[:2])]
    bad += [dict(y=_across(h)), dict(y=h), dict(y=odd), dict(y=torch.empty(7, HIDDEN, dtype=BF16))]
    slots = torch.arange(12 * page, dtype=torch.int32, device=DEV)
    for change in bad:
        with pytest.raises((ValueError, LoraError)):
            block.forward(x, h, pages, 4, **change)
        torch.cuda.synchronize()
        assert torch.equal(h, before), list(change)
        k, v = cache.read(slots)
        assert not k.any() and not v.any(), list(change)
    block.forward(x, h, pages, 4, groups=good)
    torch.cuda.synchronize()
    assert not torch.equal(h, before) and cache.status() == 0


def test_a_rotary_of_another_device():
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    cache = KvCache(4, 16, KV, D, 2)
    with pytest.raises(ValueError):
        _attention(8, cache, rotary=Rotary(64, D, device="cpu"))
