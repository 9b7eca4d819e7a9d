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
