"""Calls of the 4-bit cache that follow one another on a stream without a pause: what a call reads
is what the calls ahead of it wrote."""
import numpy as np
import pytest
import torch

from oracle import kv as ref
from test_kv_gpu import _close, _ints, _np

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _full_cache(B, page, blocks, hkv, D, seed):
    """A cache whose request b owns `blocks` pages that are all written, and its block table."""
    from segmented_rank_gemm_gb300.kv import KvCache
    g = torch.Generator().manual_seed(seed)
    n = B * blocks * page
    table = torch.randperm(B * blocks, generator=g).int().view(B, blocks)
    k, v = (torch.randn(n, hkv, D, generator=g).bfloat16() for _ in range(2))
    cache = KvCache(B * blocks, page, hkv, D, B)
    slots = (table.long()[:, :, None] * page + torch.arange(page)).reshape(-1).int()
    cache.append(k.to(DEV), v.to(DEV), slots.to(DEV))
    held = [ref.held(_np(x)).reshape(B, blocks * page, hkv, D) for x in (k, v)]
    return cache, table.to(DEV), held


@pytest.mark.parametrize("B,page,blocks,top,rounds", [(9, 256, 3, 60, 24), (300, 64, 3, 3, 24),
                                                      (1500, 16, 2, 2, 12)])
def test_attention_right_behind_the_maps(B, page, blocks, top, rounds):
    # lengths that change from batch to batch, the same arrays every time, nothing between the two
    # calls: results are those of the same calls waited for one by one
    from segmented_rank_gemm_gb300.kv import lora_kv_maps
    hkv, G, D = 2, 4, 64
    cache, table, (hk, hv) = _full_cache(B, page, blocks, hkv, D, B)
    rng = np.random.default_rng(B)
    new = rng.integers(0, top + 1, (rounds, B))
    # (an end on the page that the length is on: the batch takes no pages)
    on = rng.integers(0, blocks, (rounds, B)) * page
    lens = on + 1 + rng.integers(0, page - top, (rounds, B))
    T = int(new.sum(1).max()) + 5
    q = torch.randn(rounds, T, hkv * G, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    qd, lens_d, new_d = q.to(DEV), _ints(lens), _ints(new)
    n_free, free = _ints([0]), _ints([0])
    fill = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    kv_len, off, pos, slot, ad, counts = fill(B), fill(B + 1), fill(T), fill(T), fill(T), fill(5)

    def batch(i, out):
        lora_kv_maps(lens_d[i], new_d[i], None, page, table, free, n_free, kv_len, off, pos, slot,
                     ad, counts)
        cache.attend(qd[i], off, kv_len, table, top, out=out)

    apart, behind = torch.full_like(qd, 3.0), torch.full_like(qd, 5.0)
    for i in range(rounds):
        torch.cuda.synchronize()
        batch(i, apart[i])
        torch.cuda.synchronize()
        assert counts.tolist() == [int(new[i].sum()), 0, 0, 0, 0]
    for i in range(rounds):
        batch(i, behind[i])
    torch.cuda.synchronize()
    assert cache.status() == 0
    assert torch.equal(apart, behind)
    i = rounds - 1
    first = np.concatenate(([0], np.cumsum(new[i])))
    some = range(B) if B < 50 else range(0, B, 29)
    for b in some:
        n, m = int(lens[i, b] + new[i, b]), int(new[i, b])
        want = ref.attend(_np(q[i, first[b]:first[b] + m]), hk[b, :n], hv[b, :n], D ** -0.5)
        _close(behind[i, first[b]:first[b] + m], want, np.abs(hv).max(), "request %d" % b)
    assert not behind[i, first[-1]:].any()
    cache.close()


@pytest.mark.parametrize("new", [[1, 2, 1], [9, 12, 10]])  # few rows a cache head, many
def test_offsets_whose_difference_passes_32_bits(new):
    # from 2^31 - 1 down to -2^31 is 1 in 32 bits: still offsets out of range
    from segmented_rank_gemm_gb300.lora import LORA_EID
    from test_kv_gpu import Setup
    kv = [40, 70, 33]
    s = Setup(kv, 64, 1, 16, seed=31)
    q = s.queries(new, 4)
    top, T = max(new), sum(new)
    good = s.attend(q.to(DEV), new)
    off = np.concatenate(([0], np.cumsum(new)))
    for first, last in ((2 ** 31 - 1, -2 ** 31), (2 ** 31 - 1, -2 ** 31 + top - 1),
                        (T + 1, T + 2), (2 ** 31 - 2, 2 ** 31 - 1), (-2 ** 31, -2 ** 31 + 1)):
        bad = off.copy()
        bad[1], bad[2] = first, last  # request 1 between them; 0 and 2 end and begin there
        out = s.cache.attend(q.to(DEV), _ints(bad), _ints(kv), _ints(s.table), top)
        assert out.shape == good.shape
        assert s.cache.status() == LORA_EID
    assert torch.equal(s.attend(q.to(DEV), new), good)
    assert s.cache.status() == 0


def test_calls_after_a_wait_that_gave_up():
    # few groups over long contexts, which several CTAs share and the last to arrive joins: what was
    # counted when a wait gave up must not count for them
    from segmented_rank_gemm_gb300.lora import LORA_ETIMEOUT, LORA_OK
    from test_kv_gpu import Setup
    kv, new = [6000, 9000], [70, 1]  # many rows a cache head, few
    s = Setup(kv, 128, 1, 64, seed=32)
    q = s.queries(new, 4)
    args = q.to(DEV), _ints([0, 70, 71]), _ints(kv), _ints(s.table), 70
    want = s.cache.attend(*args)
    _close(want, s.expected(q, new, 128 ** -0.5), np.abs(s.hv).max())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side):
        s.cache.wait_selftest(stream)
        assert s.cache.status(stream) == LORA_ETIMEOUT
        assert s.cache.status(stream) == LORA_OK
        for _ in range(3):
            out = torch.zeros_like(want)
            torch.cuda.synchronize()
            s.cache.attend(*args, out=out, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert s.cache.status(stream) == LORA_OK
