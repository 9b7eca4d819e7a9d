"""The 4-bit key/value cache, the attention over it and the batch maps on the GPU, through the
public binding, against the plain 64-bit definitions of ``oracle.kv``.

Tolerances.  Maps and cached values are exact.  Attention, on the values the cache holds: the
output is rounded to bf16 once (half a step, at most 2^-8 of it); a probability is rounded to fp16 (2^-11 of it)
under a sum taken before that rounding, which moves the output by at most 2^-11 max|v|; and a
score's fp32 error, at most 2^-22 of scale * sum|q k|, moves it by that times max|v|, which is
below 2^-11 max|v| for sums up to 2^11.  Together |err| <= 2^-8 |o| + 2^-10 max|v|.
"""
import numpy as np
import pytest
import torch

from oracle import kv as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _np(t):
    return t.detach().float().cpu().numpy()


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Setup:
    """A cache filled through ``append`` with random keys and values of every request, its block
    table over shuffled pages, and the values it holds by definition."""

    def __init__(self, kv, D, hkv, page, seed=0, k_scale=1.0, v_scale=1.0, spread=1.0, shift=0.0,
                 max_requests=None):
        from segmented_rank_gemm_gb300.kv import KvCache
        self.kv, self.D, self.hkv, self.page = kv, D, hkv, page
        g = torch.Generator().manual_seed(seed)
        blocks = [-(-n // page) for n in kv]
        pages = sum(blocks) + 2
        order = torch.randperm(pages, generator=g).numpy()
        self.table = np.full((len(kv), max(blocks + [1]) + 1), 2 ** 30, np.int32)  # unread: invalid
        at = 0
        for b, n in enumerate(blocks):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = KvCache(pages, page, hkv, D, max_requests or len(kv), k_scale, v_scale)
        T = sum(kv)
        self.k = ((torch.randn(T, hkv, D, generator=g) + shift) * spread).bfloat16()
        self.v = (torch.randn(T, hkv, D, generator=g) * 0.7).bfloat16()
        slots = [self.table[b, p // page] * page + p % page for b, n in enumerate(kv)
                 for p in range(n)]
        self.slots = _ints(np.array(slots, np.int64).astype(np.int32))
        self.cache.append(self.k.to(DEV), self.v.to(DEV), self.slots)
        self.hk, self.hv = ref.held(_np(self.k), k_scale), ref.held(_np(self.v), v_scale)

    def queries(self, new, G, seed=1, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        return (torch.randn(sum(new), self.hkv * G, self.D, generator=g) * spread).bfloat16()

    def expected(self, q, new, scale, rows=None):
        out, k0, q0 = [], 0, 0
        for n, m in zip(self.kv, new):
            out.append(ref.attend(_np(q[q0:q0 + m]), self.hk[k0:k0 + n], self.hv[k0:k0 + n], scale))
            k0, q0 = k0 + n, q0 + m
        return np.concatenate(out)

    def attend(self, q, new, scale=None, out=None, max_q=None, table=None, stream=None):
        off = np.concatenate(([0], np.cumsum(new)))
        return self.cache.attend(q, _ints(off), _ints(self.kv),
                                 _ints(self.table if table is None else table),
                                 max_q or max(max(new), 1), scale, out, stream)


def _close(got, want, vmax, what=""):
    got = _np(got).astype(np.float64)
    assert got.shape == want.shape
    assert np.isfinite(got).all(), what
    lim = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * vmax
    err = np.abs(got - want)
    assert (err <= lim).all(), "%s: worst %.3g over" % (what, float((err - lim).max()))


# ---------------------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,hkv", [(16, 1), (32, 3), (64, 8), (256, 2)])
@pytest.mark.parametrize("g", [1.0, 0.03])
def test_cached_values_are_exact(D, page, hkv, g):
    from segmented_rank_gemm_gb300.kv import KvCache
    T, pages = 77, 12
    gen = torch.Generator().manual_seed(D + page)
    k = (torch.randn(T, hkv, D, generator=gen) * torch.exp(3 * torch.randn(T, 1, 1, generator=gen)))
    v = torch.randn(T, hkv, D, generator=gen) * 0.02
    k[0], v[1, :, :GROUPS] = 0, 0                 # zero groups
    k[2], v[2] = 1e-7, 1e30                       # below and above every scale
    k[3, :, 5], v[3, :, 7] = float("nan"), float("inf")
    k[4, :, 3], k[4, :, 4] = float("-inf"), float("nan")
    k[5] = torch.arange(D) % 15 - 7.0             # ties: every code and half code
    k[6] = (torch.arange(D) % 29 - 14.0) / 2
    k[6, :, ::16] = 7.0
    k, v = k.bfloat16(), v.bfloat16()
    slots = torch.randperm(pages * page, generator=gen)[:T].int()
    slots[10], slots[11] = -1, -1
    cache = KvCache(pages, page, hkv, D, 1, g, 2 * g)
    cache.append(k.to(DEV), v.to(DEV), slots.to(DEV))
    gk, gv = cache.read(slots.to(DEV))
    assert cache.status() == 0
    for got, x, s in ((gk, k, g), (gv, v, 2 * g)):
        want = torch.from_numpy(ref.held(_np(x), s).astype(np.float32)).bfloat16()
        want[10:12] = 0
        assert torch.equal(got.cpu(), want)
    # everything else is still zero
    rest = torch.from_numpy(np.setdiff1d(np.arange(pages * page), slots.numpy())).int()
    rk, rv = cache.read(rest.to(DEV))
    assert not rk.any() and not rv.any()
    cache.close()


@pytest.mark.parametrize("g", [1.0, 0.013, 1 / 3, 1.9, 3e-30, 5e30, 2e-38])
def test_quotients_at_every_tie(g):
    # values on and beside the half codes of scales of every size: n + 1/2 times the scale in bf16,
    # one bf16 step to both sides of it, and random ones
    from segmented_rank_gemm_gb300.kv import KvCache
    rng = np.random.default_rng(17)
    D, hkv, T = 128, 1, 2048
    top = (7.0 * g * np.exp2(rng.uniform(-8, 8, (T, D // 16, 1)))).astype(np.float32)
    scale = ref.to_e4m3(top / (np.float32(7) * np.float32(g))) * g
    x = scale * (rng.integers(-7, 7, (T, D // 16, 16)) + 0.5)
    x = torch.from_numpy(x.astype(np.float32)).bfloat16()
    x = (x.view(torch.int16) + torch.from_numpy(rng.integers(-1, 2, x.shape).astype(np.int16))).view(
        torch.bfloat16)
    some = torch.from_numpy(rng.random(x.shape) < 0.2)
    x = torch.where(some, torch.from_numpy((top * rng.uniform(-1, 1, x.shape)).astype(np.float32)).bfloat16(), x)
    x[:, :, 3] = torch.from_numpy(top[:, :, 0]).bfloat16()
    x = x.reshape(T, hkv, D)
    cache = KvCache(T // 16, 16, hkv, D, 1, g, g)
    slots = _ints(rng.permutation(T))
    cache.append(x.to(DEV), x.flip(-1).contiguous().to(DEV), slots)
    gk, gv = cache.read(slots)
    assert cache.status() == 0
    for got, y in ((gk, x), (gv, x.flip(-1))):
        want = torch.from_numpy(ref.held(_np(y), g).astype(np.float32)).bfloat16()
        assert torch.equal(got.cpu(), want)
    cache.close()


GROUPS = 16


def test_append_takes_strided_rows_and_flags_bad_slots():
    from segmented_rank_gemm_gb300.kv import KvCache
    from segmented_rank_gemm_gb300.lora import LORA_EID
    hkv, D, T = 2, 128, 9
    both = torch.randn(T, 3 * hkv * D, generator=torch.Generator().manual_seed(0)).bfloat16().to(DEV)
    k = both[:, hkv * D:2 * hkv * D].view(T, hkv, D)
    v = both[:, 2 * hkv * D:].view(T, hkv, D)
    cache = KvCache(4, 16, hkv, D, 1)
    slots = _ints([5, 6, 64, 7, -1, -2, 63, 0, 8])  # 64 and -2 are outside
    cache.append(k, v, slots)
    assert cache.status() == LORA_EID
    assert cache.status() == 0
    good = _ints([5, 6, -1, 7, -1, -1, 63, 0, 8])
    gk, gv = cache.read(good)
    for got, x in ((gk, k), (gv, v)):
        want = torch.from_numpy(ref.held(_np(x)).astype(np.float32)).bfloat16()
        want[[2, 4, 5]] = 0
        assert torch.equal(got.cpu(), want)
    cache.read(slots)
    assert cache.status() == LORA_EID
    cache.append(k[:0], v[:0], slots[:0])
    cache.close()


# ---------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------

EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 100, 127, 128, 129, 255, 256, 300]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 11, 16])
@pytest.mark.parametrize("page", [16, 64])
def test_single_tokens(D, G, page):
    s = Setup(EDGES, D, 2, page, seed=D + G + page)
    new = [1] * len(EDGES)
    q = s.queries(new, G)
    out = s.attend(q.to(DEV), new)
    assert s.cache.status() == 0
    _close(out, s.expected(q, new, D ** -0.5), np.abs(s.hv).max())


@pytest.mark.parametrize("D,G,page", [(64, 1, 32), (64, 4, 16), (128, 4, 64), (128, 8, 128),
                                      (128, 5, 16), (64, 40, 256)])
def test_ragged_queries(D, G, page):
    # prompts from nothing, behind a context, ending inside pages and tiles; idle requests;
    # fewer positions than queries (the first rows see nothing)
    kv = [1, 5, 64, 65, 200, 33, 0, 7, 3, 130, 16, 0]
    new = [1, 5, 64, 1, 70, 2, 0, 0, 6, 129, 8, 2]
    s = Setup(kv, D, 2, page, seed=3)
    q = s.queries(new, G)
    out = s.attend(q.to(DEV), new)
    assert s.cache.status() == 0
    want = s.expected(q, new, D ** -0.5)
    _close(out, want, np.abs(s.hv).max())
    first = sum(new[:8])
    assert not out[first:first + 3].any()  # rows 0..2 of the request with 3 positions, 6 rows
    assert not out[-2:].any()


def test_prompt_of_some_length():
    kv, new = [700, 40, 513], [400, 40, 257]
    s = Setup(kv, 128, 1, 64, seed=4)
    q = s.queries(new, 4)
    out = s.attend(q.to(DEV), new)
    _close(out, s.expected(q, new, 128 ** -0.5), np.abs(s.hv).max())


@pytest.mark.parametrize("D,G,kv,new", [
    (128, 4, [6000], [70]), (128, 8, [300, 9000, 5, 2600], [300, 33, 5, 40]),
    (64, 4, [20000, 64], [9, 64]), (128, 1, [4000, 3000, 3500], [300, 17, 260])])
def test_long_prompts_are_cut_and_joined(D, G, kv, new):
    # few groups over long contexts: a group's tiles are shared by several CTAs
    s = Setup(kv, D, 1, 64, seed=21)
    q = s.queries(new, G)
    out = s.attend(q.to(DEV), new)
    assert s.cache.status() == 0
    _close(out, s.expected(q, new, D ** -0.5), np.abs(s.hv).max())
    assert torch.equal(out, s.attend(q.to(DEV), new))


@pytest.mark.parametrize("B,hi,top", [(12, 400, 1500), (700, 12, 120), (2100, 8, 40)])
def test_prompts_of_many_lengths(B, hi, top):
    # groups of very different sizes, requests of few rows and none between them, more requests
    # than a CTA has threads
    rng = np.random.default_rng(B)
    new = [int(n) for n in rng.integers(0, hi + 1, B)]
    kv = [n + int(rng.integers(0, top)) for n in new]
    s = Setup(kv, 64, 2, 32, seed=22)
    q = s.queries(new, 4)
    out = s.attend(q.to(DEV), new)
    assert s.cache.status() == 0
    _close(out, s.expected(q, new, 0.125), np.abs(s.hv).max())
    assert torch.equal(out, s.attend(q.to(DEV), new))


@pytest.mark.parametrize("kv", [[60000], [1, 50000, 3, 17000]])
def test_long_contexts_are_split_and_joined(kv):
    s = Setup(kv, 128, 1, 64, seed=5, spread=1.5)
    new = [1] * len(kv)
    q = s.queries(new, 4)
    out = s.attend(q.to(DEV), new)
    _close(out, s.expected(q, new, 128 ** -0.5), np.abs(s.hv).max())
    again = s.attend(q.to(DEV), new)
    assert torch.equal(out, again)


def test_many_requests():
    rng = np.random.default_rng(6)
    kv = [int(n) for n in rng.integers(0, 90, 700)]
    new = [int(rng.integers(0, 3)) if n > 2 else min(n, 1) for n in kv]
    s = Setup(kv, 64, 2, 32, seed=6)
    q = s.queries(new, 2)
    out = s.attend(q.to(DEV), new)
    _close(out, s.expected(q, new, 0.125), np.abs(s.hv).max())


@pytest.mark.parametrize("spread,shift,scale", [(6.0, 0.0, None), (1.0, 40.0, None),
                                                (3.0, 0.0, -0.2), (1.0, 0.0, 0.0)])
def test_extreme_scores(spread, shift, scale):
    # scores far apart (one position takes all), far from zero, turned over, or all equal; growing
    # along the context so that the running reference moves again and again.  The products'
    # sums exceed 2^11 here, so queries are cut to a few dimensions, which keeps them below.
    kv = [333, 1000]
    s = Setup(kv, 128, 1, 64, seed=7, spread=spread, shift=shift)
    new = [1, 2]
    q = s.queries(new, 4, spread=2.0)
    q[:, :, 8:] = 0
    out = s.attend(q.to(DEV), new, scale)
    _close(out, s.expected(q, new, 128 ** -0.5 if scale is None else scale), np.abs(s.hv).max())


def test_growing_scores_move_the_reference():
    s = Setup([2000], 128, 1, 64, seed=8)
    # keys along one dimension, growing: score of position j about j / 8 in units of log2(e)
    k = torch.zeros(2000, 1, 128)
    k[:, 0, 0] = torch.arange(2000) / 16.0
    v = s.v
    s.cache.append(k.bfloat16().to(DEV), v.to(DEV), s.slots)
    s.hk = ref.held(_np(k.bfloat16()))
    q = torch.zeros(1, 4, 128)
    q[0, :, 0] = torch.tensor([1.0, -1.0, 4.0, 0.25])
    q = q.bfloat16()
    out = s.attend(q.to(DEV), [1], 1.0)
    _close(out, s.expected(q, [1], 1.0), np.abs(s.hv).max())


def test_scales_of_the_cache():
    s = Setup([200, 31], 128, 2, 32, seed=9, k_scale=0.01, v_scale=25.0, spread=0.02)
    q = s.queries([1, 4], 4, spread=20.0)
    out = s.attend(q.to(DEV), [1, 4])
    _close(out, s.expected(q, [1, 4], 128 ** -0.5), np.abs(s.hv).max())


def test_nan_and_infinite_queries_stay_in_their_rows():
    kv, new = [90, 70], [1, 20]
    s = Setup(kv, 128, 1, 64, seed=10)
    q = s.queries(new, 4)
    want = s.expected(q, new, 128 ** -0.5)
    bad = q.clone()
    bad[3, 2, 17] = float("nan")
    bad[5, 0, 3] = float("inf")
    out = _np(s.attend(bad.to(DEV), new))
    assert np.isnan(out[3, 2]).all()
    mask = np.ones(out.shape[:2], bool)
    mask[3, 2] = mask[5, 0] = False
    _close(torch.from_numpy(out[mask]), want[mask], np.abs(s.hv).max())


def test_strided_rows_padding_and_rows_outside():
    kv, new = [40, 80], [1, 33]
    s = Setup(kv, 128, 2, 64, seed=11)
    G, T = 4, 34
    q = s.queries(new, G)
    width = 2 * G * 128
    wide = torch.full((T + 6, width + 264), 9.0, dtype=torch.bfloat16, device=DEV)
    qv = wide[:, 8:8 + width].view(T + 6, 2 * G, 128)
    qv[:T] = q.to(DEV)
    outw = torch.full((T + 6, width + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    out = outw[:, :width].view(T + 6, 2 * G, 128)
    s.attend(qv, new, out=out)
    _close(out[:T], s.expected(q, new, 128 ** -0.5), np.abs(s.hv).max())
    assert not out[T:].any()           # padding rows are zero
    assert (outw[:, width:] == 5).all()  # and nothing beside the rows is written


def test_on_a_stream_and_in_a_graph():
    kv, new = [300, 2], [1, 1]
    s = Setup(kv, 128, 2, 16, seed=12)
    q = s.queries(new, 4).to(DEV)
    off, lens, table = _ints([0, 1, 2]), _ints(kv), _ints(s.table)
    want = s.cache.attend(q, off, lens, table, 1)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.zeros_like(q)
    s.cache.attend(q, off, lens, table, 1, out=out, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.attend(q, off, lens, table, 1, out=out)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_bad_tables_lengths_and_offsets_are_flagged():
    from segmented_rank_gemm_gb300.lora import LORA_EID
    kv, new = [100, 50, 60], [1, 1, 1]
    s = Setup(kv, 128, 2, 64, seed=13)
    q = s.queries(new, 4)
    want = s.expected(q, new, 128 ** -0.5)
    vmax = np.abs(s.hv).max()
    for bad in (10 ** 6, -1):
        table = s.table.copy()
        table[1, 0] = bad
        out = s.attend(q.to(DEV), new, table=table)
        assert s.cache.status() == LORA_EID
        _close(out[[0, 2]], want[[0, 2]], vmax)
    for lens in ([100, -5, 60], [100, 10 ** 6, 60]):
        # a length past the table reads its unused entries, which are invalid: still flagged
        out = s.cache.attend(q.to(DEV), _ints([0, 1, 2, 3]), _ints(lens), _ints(s.table), 1)
        assert s.cache.status() == LORA_EID
        _close(out[[0, 2]], want[[0, 2]], vmax)
    for off in ([0, 1, 5, 3], [0, 1, -4, 3], [0, 1, 0, 3]):
        s.cache.attend(q.to(DEV), _ints(off), _ints(kv), _ints(s.table), 1)
        assert s.cache.status() == LORA_EID
    # more new tokens than max_q
    s.cache.attend(q.to(DEV), _ints([0, 1, 3, 3]), _ints(kv), _ints(s.table), 1)
    assert s.cache.status() == LORA_EID
    assert s.cache.status() == 0


def test_refusals():
    from segmented_rank_gemm_gb300.kv import KvCache
    from segmented_rank_gemm_gb300.lora import LoraError
    for args in ((0, 16, 1, 64, 1), (4, 24, 1, 64, 1), (4, 16, 0, 64, 1), (4, 16, 1, 96, 1),
                 (4, 16, 1, 64, 0), (2 ** 28, 16, 1, 64, 1), (4, 16, 1, 64, 1, 0.0),
                 (4, 16, 1, 64, 1, 1.0, float("inf")), (4, 512, 1, 64, 1), (4, 8, 1, 64, 1)):
        with pytest.raises(LoraError):
            KvCache(*args)
    cache = KvCache(4, 16, 2, 64, 2)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    off, lens, table = _ints([0, 1, 2]), _ints([1, 1]), _ints(np.zeros((2, 2)))
    ok = dict(q=q, q_offsets=off, kv_len=lens, block_table=table, max_q=1)
    for change in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q.cpu()), dict(max_q=0),
                   dict(q_offsets=off[:2]), dict(q_offsets=off.long()), dict(out=q),
                   dict(kv_len=_ints([1, 1, 1]), q_offsets=_ints([0, 1, 1, 2])),
                   dict(block_table=table[:1]), dict(scale=float("nan")), dict(out=q[:1]),
                   dict(q=q.transpose(0, 1)[:2]),
                   dict(q=torch.zeros(2, 4 * 64 + 4, dtype=torch.bfloat16,
                                      device=DEV)[:, :256].view(2, 4, 64))):
        with pytest.raises(LoraError):
            cache.attend(**{**ok, **change})
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    for args in ((k, k[:1], lens), (k, k, lens[:1]), (k.float(), k, lens), (k, k, lens.long())):
        with pytest.raises(LoraError):
            cache.append(*args)
    with pytest.raises(LoraError):
        cache.read(lens, k[:1], k)
    cache.attend(**ok)
    cache.attend(**{**ok, "q": q[:0], "q_offsets": _ints([0, 0, 0])})
    cache.close()


# ---------------------------------------------------------------------------------------
# block tables and slot maps
# ---------------------------------------------------------------------------------------

def _maps(lens, new, adapter, page, blocks, n_free, T, num_pages=None, seed=0, inplace=False,
          spoil=None):
    from segmented_rank_gemm_gb300.kv import lora_kv_maps
    rng = np.random.default_rng(seed)
    B = len(lens)
    used = [-(-max(a, 0) // page) for a in lens]
    num_pages = num_pages or sum(min(u, blocks) for u in used) + max(n_free, 0) + 5
    ids = rng.permutation(num_pages).astype(np.int32)
    table = np.full((B, blocks), -7, np.int32)
    at = 0
    for b, u in enumerate(used):
        u = min(u, blocks)
        table[b, :u] = ids[at:at + u]
        at += u
    free = np.full(num_pages, -9, np.int32)
    free[:max(n_free, 0)] = ids[at:at + max(n_free, 0)]
    if spoil:
        spoil(table, free)
    want = ref.maps(lens, new, adapter, page, table, free, n_free, T)
    t = {"lens": _ints(lens), "table": _ints(table), "counts": _ints([0, n_free, 0, 0, 0])}
    kv_len = t["lens"] if inplace else torch.full((B,), -3, dtype=torch.int32, device=DEV)
    n_free_t = t["counts"][1:2] if inplace else _ints([n_free])
    fill = lambda n: torch.full((n,), -3, dtype=torch.int32, device=DEV)  # noqa: E731
    off, pos, slot, ad = fill(B + 1), fill(T), fill(T), fill(T)
    lora_kv_maps(t["lens"], _ints(new), None if adapter is None else _ints(adapter), page,
                 t["table"], _ints(free), n_free_t, kv_len, off, pos, slot, ad, t["counts"])
    got = {"table": t["table"], "kv_len": kv_len, "q_offsets": off, "position": pos,
           "kv_slot": slot, "token_slot": ad, "counts": t["counts"]}
    for name, x in got.items():
        w = np.asarray(want[name])
        x = x.cpu().numpy()
        if name == "counts" and want["counts"][3]:
            assert x[3] == want["counts"][3] and list(x[:3]) == list(w[:3]) and x[4] == 0
            continue
        assert np.array_equal(x, w), name
    return want


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("inplace", [False, True])
def test_maps_small(page, inplace):
    lens = [0, 1, 15, 16, 17, 63, 64, 0, 100, 256, 0]
    new = [1, 1, 1, 1, 40, 1, 1, 0, 0, 300, 65]
    _maps(lens, new, list(range(-1, 10)), page, 40, 60, sum(new) + 3, inplace=inplace)
    _maps(lens, new, None, page, 40, 60, sum(new), inplace=inplace, seed=1)
    _maps([5], [0], [3], page, 1, 0, 0, inplace=inplace)
    _maps([0], [page], [3], page, 1, 1, page, inplace=inplace)


@pytest.mark.parametrize("B,hi,page", [(1, 70000, 16), (512, 1, 64), (3000, 30, 32), (16384, 3, 16),
                                       (1025, 100, 128)])
def test_maps_large(B, hi, page):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 400, B)]
    new = [int(x) for x in rng.integers(0, hi + 1, B)] if hi < 1000 else [hi]
    blocks = max((a + b) for a, b in zip(lens, new)) // page + 2
    for inplace in (False, True):
        _maps(lens, new, list(rng.integers(-1, 9, B)), page, blocks,
              sum(-(-b // page) + 1 for b in new), sum(new) + 11, seed=B, inplace=inplace)


@pytest.mark.parametrize("big", [False, True])
def test_maps_of_a_batch_that_does_not_fit(big):
    n = 6000 if big else 60  # several CTAs or one
    for inplace in (False, True):
        assert _maps([3, 30], [n, 1], None, 16, 4000, 2, n + 1, inplace=inplace)["counts"][3] == 2
        assert _maps([3, 30], [n, 1], None, 16, 4000, 900, n, inplace=inplace)["counts"][3] == 1
        assert _maps([3, 30], [n, 1], None, 16, 2, 900, n + 1, inplace=inplace)["counts"][3] == 1
        assert _maps([3, -1], [n, 1], None, 16, 4000, 900, n + 1, inplace=inplace)["counts"][3] == 1
        assert _maps([3, 9], [n, -1], None, 16, 4000, 900, n + 1, inplace=inplace)["counts"][3] == 1
        assert _maps([3, 2 ** 31 - 1], [n, 2 ** 31 - 1], None, 16, 4000, 900, n + 1, num_pages=9000,
                     inplace=inplace)["counts"][3] == 1
        assert _maps([3, 9], [n, 1], None, 16, 4000, -1, n + 1, inplace=inplace)["counts"][3] == 2


@pytest.mark.parametrize("n", [40, 9000])
def test_maps_with_bad_page_ids(n):
    def spoil(table, free):
        table[0, 2] = 2 ** 28  # its slots pass 2^31
        table[1, 0] = -1
        free[580] = -5
    w = _maps([40, 3, 0], [20, 2, n], [1, 2, 3], 16, 600, 600, n + 30, spoil=spoil)
    assert w["counts"][3] == 4


def test_release_returns_pages_in_order():
    from segmented_rank_gemm_gb300.kv import PageTable
    rng = np.random.default_rng(0)
    B, page, pages = 300, 16, 4000
    t = PageTable(pages, page, B, 40, 20000)
    new = rng.integers(0, 60, B)
    t.step(_ints(new), _ints(rng.integers(0, 5, B)))
    tokens, free, taken, flags, _ = t.status()
    need = int(sum(-(-x // page) for x in new))
    assert (tokens, free, taken, flags) == (int(new.sum()), pages - need, need, 0)
    table, stack = t.block_table.cpu().numpy(), t.free_pages.cpu().numpy().copy()
    done = rng.integers(0, 2, B)
    t.release(_ints(done))
    want = [int(table[b, j]) for b in range(B) if done[b] for j in range(-(-new[b] // page))]
    assert t.status()[4] == 0 and int(t.n_free) == free + len(want)
    assert t.free_pages.cpu().tolist()[:free + len(want)] == stack[:free].tolist() + want
    assert t.kv_len.cpu().tolist() == [0 if done[b] else int(new[b]) for b in range(B)]
    # a second step takes them again, from the top
    t.step(_ints(np.where(done, 1, 0)))
    assert t.status()[2] == int(done.sum())
    first = t.block_table[int(np.flatnonzero(done)[0]), 0].item()
    assert first == want[-1]


def test_release_refuses_what_cannot_be():
    from segmented_rank_gemm_gb300.kv import lora_kv_release
    table, free = _ints(np.arange(8).reshape(2, 4)), _ints(np.zeros(5))
    for lens, n_free, code in (([-1, 3], 0, 1), ([65, 3], 0, 1), ([64, 64], 0, 2), ([16, 16], 4, 2),
                               ([1, 1], -1, 2), ([64, 0], 1, 0)):
        L, n, st = _ints(lens), _ints([n_free]), _ints([9])
        lora_kv_release(_ints([1, 1]), L, 16, table, free, n, st)
        assert int(st) == code
        assert L.tolist() == ([0, 0] if code == 0 else lens)
        assert int(n) == (5 if code == 0 else n_free)


def test_maps_refusals():
    from segmented_rank_gemm_gb300.kv import PageTable
    from segmented_rank_gemm_gb300.lora import LoraError
    t = PageTable(10, 16, 4, 3, 8)
    for new in (_ints([1, 1, 1]), _ints([1] * 4).long(), _ints([1] * 4).cpu()):
        with pytest.raises(LoraError):
            t.step(new)
    with pytest.raises(LoraError):
        t.release(_ints([1, 1, 1]))
    t.page_size = 20
    with pytest.raises(LoraError):
        t.step(_ints([1] * 4))


def test_pages_through_steps_and_a_graph():
    """A few captured steps through PageTable, append and attend, with requests finishing."""
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable
    B, page, hkv, G, D = 5, 16, 2, 2, 64
    table = PageTable(60, page, B, 8, 64)
    cache = KvCache(60, page, hkv, D, B)
    gen = torch.Generator().manual_seed(1)
    held_k, held_v = [[] for _ in range(B)], [[] for _ in range(B)]
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    T = 64
    k = torch.zeros(T, hkv, D, dtype=torch.bfloat16, device=DEV)
    v, q = torch.zeros_like(k), torch.zeros(T, hkv * G, D, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(q)

    def step():
        table.step(new)
        cache.append(k, v, table.kv_slot)
        cache.attend(q, table.q_offsets, table.kv_len, table.block_table, T, out=out)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i, counts in enumerate([[20, 3, 0, 17, 1], [1, 1, 30, 0, 1], [1, 1, 1, 1, 1], [2, 0, 15, 16, 8]]):
        n = sum(counts)
        new.copy_(_ints(counts))
        kk, vv, qq = (torch.randn(T, h, D, generator=gen).bfloat16() for h in (hkv, hkv, hkv * G))
        k.copy_(kk), v.copy_(vv), q.copy_(qq)
        graph.replay()
        torch.cuda.synchronize()
        assert table.status()[0] == n and table.status()[3] == 0 and cache.status() == 0
        at = 0
        for b, c in enumerate(counts):
            held_k[b] += list(ref.held(_np(kk[at:at + c])))
            held_v[b] += list(ref.held(_np(vv[at:at + c])))
            if c:
                want = ref.attend(_np(qq[at:at + c]), np.array(held_k[b]), np.array(held_v[b]), D ** -0.5)
                _close(out[at:at + c], want, 3.5, "step %d request %d" % (i, b))
            at += c
        assert not out[n:].any()
        if i == 1:
            table.release(_ints([0, 1, 0, 1, 0]))
            held_k[1], held_v[1], held_k[3], held_v[3] = [], [], [], []
