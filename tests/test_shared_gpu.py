"""Attention of requests that share prefixes, and to an encoder's states, over the 4-bit cache on
the GPU, against the plain 64-bit definitions of ``oracle.kv``.

Tolerances: those of attention over the cache (one rounding of the output to bf16, 2^-8 of it;
probabilities rounded to fp16 under an exact sum, 2^-11 max|v|; scores in fp32, below that):
2^-8 |o| + 2^-10 max|v|.  Joining two parts is a weighted mean in fp32, whose weights sum to one:
it adds some 2^-22 max|v|, which that leaves room for.
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


def _close(got, want, vmax, what=""):
    got = _np(got).astype(np.float64)
    assert got.shape == want.shape
    assert np.isfinite(got).all(), what
    err, lim = np.abs(got - want), 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * vmax
    assert (err <= lim).all(), "%s: worst %.3g over" % (what, float((err - lim).max()))


class Batch:
    """Groups of requests: ``groups`` lists (prefix positions, [(own positions, new tokens)]); the
    prefix's pages are in a table row of its own behind the requests', or (``leader``) in its first
    member's.  ``alone``: requests attended by themselves (shared_len 0) although they are members."""

    def __init__(self, groups, D, hkv, G, page, seed=0, leader=False, alone=(), outside=(), spread=1.0):
        from segmented_rank_gemm_gb300.kv import KvCache
        self.D, self.hkv, self.G, self.page = D, hkv, G, page
        g = torch.Generator().manual_seed(seed)
        self.first, self.prefix_row, self.prefix_len, self.new, self.kv, self.shared = [0], [], [], [], [], []
        runs, rows = [], []  # runs of positions with pages of their own; the runs of each request
        B = sum(len(m) for _, m in groups) + len(outside)
        for i, (prefix, members) in enumerate(groups):
            runs.append(prefix)
            prefix_run = len(runs) - 1
            self.prefix_row.append(self.first[-1] if leader else B + i)
            self.prefix_len.append(prefix)
            for own, new in members:
                runs.append(own)
                rows.append((prefix_run, len(runs) - 1))
                self.shared.append(0 if len(self.kv) in alone else prefix)
                self.kv.append(prefix + own)
                self.new.append(new)
            self.first.append(len(self.kv))
        for own, new in outside:  # in no group
            runs.append(own)
            rows.append((None, len(runs) - 1))
            self.shared.append(0)
            self.kv.append(own)
            self.new.append(new)
        self.B, count = B, [-(-n // page) for n in runs]
        pages = sum(count) + 2
        order = torch.randperm(pages, generator=g).numpy()
        at = np.concatenate(([0], np.cumsum(count)))
        ids = [order[at[i]:at[i + 1]] for i in range(len(runs))]
        wide = max(-(-n // page) for n in self.kv + [1]) + 1
        self.table = np.full((B + len(groups), wide), 2 ** 30, np.int32)  # unread: invalid
        where = []
        for b, (p, o) in enumerate(rows):
            row = np.concatenate((ids[p] if p is not None else ids[0][:0], ids[o]))
            self.table[b, :len(row)] = row
        for i, row in enumerate(self.prefix_row):
            run = [k for k, (p, _) in enumerate(groups)][i]
            prefix_run = sum(1 + len(m) for _, m in groups[:run])
            self.table[row, :count[prefix_run]] = ids[prefix_run]
        T = sum(runs)
        k = (torch.randn(T, hkv, D, generator=g) * spread).bfloat16()
        v = (torch.randn(T, hkv, D, generator=g) * 0.7).bfloat16()
        for i, n in enumerate(runs):
            where += [int(ids[i][p // page]) * page + p % page for p in range(n)]
        self.cache = KvCache(pages, page, hkv, D, B + len(groups))
        self.cache.append(k.to(DEV), v.to(DEV), _ints(where))
        hk, hv = ref.held(_np(k)), ref.held(_np(v))
        start = np.concatenate(([0], np.cumsum(runs)))
        cut = [slice(start[i], start[i + 1]) for i in range(len(runs))]
        self.keys = [tuple(np.concatenate(([x[cut[p]]] if p is not None else []) + [x[cut[o]]])
                           for x in (hk, hv)) for p, o in rows]
        self.vmax = np.abs(hv).max()
        self.q = torch.randn(sum(self.new), hkv * G, D, generator=g).bfloat16()
        self.offsets = np.concatenate(([0], np.cumsum(self.new)))
        self.scale = D ** -0.5

    def expected(self, q=None):
        q = _np(self.q if q is None else q)
        return np.concatenate([ref.attend(q[a:b], k, v, self.scale)
                               for a, b, (k, v) in zip(self.offsets, self.offsets[1:], self.keys)])

    def args(self, **change):
        """kv_len and the table have a row for every prefix behind the requests' where they need it."""
        a = dict(q=self.q.to(DEV), q_offsets=np.concatenate((self.offsets, [self.offsets[-1]] * (len(self.table) - self.B))),
                 kv_len=self.kv + [0] * (len(self.table) - self.B), block_table=self.table,
                 max_q=max(max(self.new), 1), group_offsets=self.first, prefix_row=self.prefix_row,
                 prefix_len=self.prefix_len, shared_len=self.shared + [0] * (len(self.table) - self.B))
        a.update(change)
        return {k: _ints(v) if isinstance(v, (list, np.ndarray)) else v for k, v in a.items()}

    def attend(self, **change):
        return self.cache.attend_shared(**self.args(**change))

    def check(self, **more):
        out = self.attend(**more)
        assert self.cache.status() == 0
        _close(out, self.expected(), self.vmax)
        assert torch.equal(out, self.attend(**more))
        return out


# ---------------------------------------------------------------------------------------
# shared prefixes
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("D,G,page", [(64, 1, 16), (128, 4, 64), (64, 3, 32), (128, 8, 16), (128, 5, 128),
                                      (64, 11, 256)])
def test_single_tokens(D, G, page):
    # prefixes of one page and of many; members of few rows and of many; own positions up to and
    # past a page's and a tile's end, down to the new token alone
    rng = np.random.default_rng(D + G)
    groups = [(page, [(1, 1), (2, 1)]), (3 * page, [(n, 1) for n in (1, 15, 16, 17, 31, 33, 64, 65, 100)]),
              (7 * page, [(40, 1)]), (20 * page, [(int(rng.integers(1, 90)), 1) for _ in range(70)])]
    Batch(groups, D, 2, G, page, seed=G).check()


@pytest.mark.parametrize("leader", [False, True])
@pytest.mark.parametrize("D,G,page", [(128, 4, 16), (64, 2, 64)])
def test_several_tokens_idle_members_and_requests_by_themselves(D, G, page, leader):
    groups = [(2 * page, [(3, 3), (50, 7), (9, 1), (130, 64)]), (0, [(5, 5), (70, 1)]),
              (5 * page, [(4, 0), (0, 0)]), (4 * page, [(9, 2), (33, 5), (80, 80), (7, 1)]),
              (page, [(1, 1)])]
    b = Batch(groups, D, 2, G, page, seed=3, leader=leader, alone=(2, 9), outside=[(20, 2), (0, 0), (300, 1)])
    b.check()


@pytest.mark.parametrize("prefix,members,G,D", [(20000, 3, 4, 128), (30016, 40, 4, 128), (9008, 2, 1, 64),
                                                (6000, 300, 2, 64)])
def test_long_prefixes_are_cut_and_joined(prefix, members, G, D):
    rng = np.random.default_rng(prefix)
    groups = [(prefix // 16 * 16, [(int(rng.integers(1, 60)), 1) for _ in range(members)])]
    Batch(groups, D, 1, G, 16, seed=8, spread=1.4).check()


def test_prompts_that_share():
    groups = [(512, [(300, 300), (20, 20), (513, 257)]), (1024, [(700, 64), (1, 1)])]
    Batch(groups, 128, 1, 4, 64, seed=5).check()


def test_many_groups_and_requests():
    rng = np.random.default_rng(6)
    groups = [(int(rng.integers(0, 9)) * 32, [(int(n), int(min(n, rng.integers(0, 3))))
                                             for n in rng.integers(1, 40, rng.integers(1, 12))])
              for _ in range(150)]
    Batch(groups, 64, 2, 2, 32, seed=6).check()


def test_all_requests_by_themselves_is_attend():
    groups = [(64, [(30, 1), (50, 4)]), (128, [(9, 9)])]
    b = Batch(groups, 128, 2, 4, 16, alone=(0, 1, 2))
    a = b.args()
    out = b.cache.attend_shared(**a)
    for k in ("group_offsets", "prefix_row", "prefix_len", "shared_len"):
        del a[k]
    assert torch.equal(out, b.cache.attend(**a))


@pytest.mark.parametrize("wide", [0, 4000])
def test_small_batches_on_both_sides_of_the_rule(wide):
    # a wider table (whose entries are not read) makes the longest request possible longer
    b = Batch([(64, [(30, 1), (50, 4), (1, 1)]), (128, [(9, 2)])], 128, 2, 2, 16, seed=4)
    table = np.concatenate((b.table, np.full((len(b.table), wide), 2 ** 30, np.int32)), 1)
    b.check(block_table=table)
    shared = b.shared + [0, 0]
    from segmented_rank_gemm_gb300.lora import LORA_EID
    for change in (dict(shared_len=[64, 32] + shared[2:]), dict(prefix_len=[32, 128]), dict(group_offsets=[0, 2, 4])):
        b.attend(block_table=table, **change)
        assert b.cache.status() == LORA_EID


def test_scores_far_apart_between_prefix_and_own_positions():
    # all of the weight in the prefix, all of it behind, and both
    b = Batch([(320, [(40, 1), (33, 2), (64, 1)])], 128, 1, 4, 16, seed=11, spread=6.0)
    q = b.q * 2
    q[:, :, 8:] = 0
    out = b.attend(q=q.to(DEV))
    _close(out, b.expected(q), b.vmax)


def test_nan_queries_stay_in_their_rows():
    b = Batch([(64, [(10, 1), (20, 1), (30, 12)])], 128, 2, 4, 16, seed=12)
    want = b.expected()
    bad = b.q.clone()
    bad[1, 2, 17] = float("nan")
    out = _np(b.attend(q=bad.to(DEV)))
    assert np.isnan(out[1, 2]).all()
    mask = np.ones(out.shape[:2], bool)
    mask[1, 2] = False
    _close(torch.from_numpy(out[mask]), want[mask], b.vmax)


def test_strided_rows_padding_streams_and_a_graph():
    b = Batch([(256, [(10, 1), (20, 3), (30, 1)]), (64, [(5, 1)] * 9)], 64, 2, 4, 64, seed=13)
    want, T, width = b.expected(), sum(b.new), 8 * 64
    wide = torch.full((T + 5, width + 64), 9.0, dtype=torch.bfloat16, device=DEV)
    q = wide[:, 8:8 + width].view(T + 5, 8, 64)
    q[:T] = b.q.to(DEV)
    outw = torch.full((T + 5, width + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    out = outw[:, :width].view(T + 5, 8, 64)
    ws = b.cache.shared_workspace(T + 5, 8)
    ws.view(torch.float32).fill_(float("nan"))
    a = b.args(q=q, out=out, workspace=ws)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.cache.attend_shared(**a, stream=stream)
    stream.synchronize()
    _close(out[:T], want, b.vmax)
    assert not out[T:].any() and (outw[:, width:] == 5).all()
    once = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.cache.attend_shared(**a)
    for _ in range(3):
        out.fill_(3.0)
        ws.view(torch.float32).fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, once)


def test_calls_without_a_pause_share_a_workspace():
    # prefixes of many rows and of few in turn, each call reading what the one before wrote
    a = Batch([(2048, [(20, 1)] * 40)], 128, 2, 4, 64, seed=14)
    b = Batch([(512, [(7, 1)] * 2), (64, [(100, 1)] * 30)], 128, 2, 4, 64, seed=15)
    ws = torch.empty(a.cache.shared_workspace(40, 8).numel(), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(x.q, device=DEV) for x in (a, b)]
    args = [x.args(out=o, workspace=ws) for x, o in zip((a, b), outs)]
    for _ in range(20):
        for x, k in zip((a, b), args):
            x.cache.attend_shared(**k)
    for x, o in zip((a, b), outs):
        _close(o, x.expected(), x.vmax)
        assert x.cache.status() == 0


def test_what_cannot_be_is_flagged():
    from segmented_rank_gemm_gb300.lora import LORA_EID
    b = Batch([(64, [(20, 1), (30, 2)]), (128, [(9, 1), (40, 1)])], 64, 1, 4, 32, seed=16)
    want, shared, extra = b.expected(), list(b.shared), [0, 0]
    ok = slice(3, 5)  # rows of the second group
    bad = [dict(prefix_len=[64, 128], shared_len=[32, 64, 128, 128] + extra),  # not the group's
           dict(shared_len=[64, 96, 128, 128] + extra),   # a query would not see all of it
           dict(shared_len=[64, 70, 128, 128] + extra), dict(shared_len=[64, -32, 128, 128] + extra),
           dict(shared_len=[2 ** 30, 64, 128, 128] + extra),
           dict(prefix_len=[63, 128]), dict(prefix_len=[-64, 128]), dict(prefix_len=[2 ** 30, 128]),
           dict(prefix_row=[-1, 5]), dict(prefix_row=[6, 5]), dict(prefix_row=[2 ** 31 - 1, 5]),
           dict(group_offsets=[1, 2, 4]), dict(group_offsets=[-1, 2, 4]), dict(group_offsets=[3, 2, 4])]
    for change in bad:
        out = b.attend(**change)
        assert b.cache.status() == LORA_EID, change
        _close(out[ok], want[ok], b.vmax, str(change))
    for change in (dict(group_offsets=[0, 2, 9]), dict(group_offsets=[0, 2 ** 31 - 1, -2 ** 31])):
        b.attend(**change)
        assert b.cache.status() == LORA_EID
    table = b.table.copy()
    table[b.prefix_row[0], 0] = 10 ** 6
    out = b.attend(block_table=table)
    assert b.cache.status() == LORA_EID
    _close(out[ok], want[ok], b.vmax)
    assert b.cache.status() == 0 and b.shared == shared
    b.check()


def test_refusals():
    from segmented_rank_gemm_gb300.lora import LoraError
    b = Batch([(16, [(2, 1), (3, 1)])], 64, 1, 4, 16)
    ok = b.args()
    ws = b.cache.shared_workspace(2, 4)
    assert ws.numel() == 2 * 4 * 8 * 66
    for change in (dict(group_offsets=ok["group_offsets"][:1]), dict(group_offsets=_ints([0, 1, 2, 2, 2])),
                   dict(prefix_row=ok["prefix_row"][:0]), dict(prefix_len=ok["prefix_len"].long()),
                   dict(shared_len=ok["shared_len"][:2]), dict(workspace=ws[:-1]), dict(workspace=ws.cpu()),
                   dict(workspace=torch.empty(ws.numel() + 8, dtype=torch.uint8, device=DEV)[8:]),
                   dict(workspace=torch.empty(ws.numel(), 2, dtype=torch.uint8, device=DEV)[:, 0]),
                   dict(max_q=0), dict(scale=float("inf")), dict(out=ok["q"])):
        with pytest.raises(LoraError):
            b.cache.attend_shared(**{**ok, **change})
    big = torch.empty(1 << 16, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(LoraError):
        b.cache.attend_shared(**{**ok, "out": big[:512].view(2, 4, 64), "workspace": big[64:].view(torch.uint8)})
    for n in ((-1, 4), (2, 0), (1 << 21, 4)):
        with pytest.raises(LoraError):
            b.cache.shared_workspace(*n)
    b.check()
    empty = {**ok, "q": ok["q"][:0], "q_offsets": _ints([0] * 4)}
    b.cache.attend_shared(**empty)


# ---------------------------------------------------------------------------------------
# an encoder's states
# ---------------------------------------------------------------------------------------

def _cross(kv, new, D, hkv, G, page, seed, spread=1.0, scale=None):
    b = Batch([(0, [(n, m) for n, m in zip(kv, new)])], D, hkv, G, page, seed, spread=spread)
    a = b.args()
    for k in ("group_offsets", "prefix_row", "prefix_len", "shared_len"):
        del a[k]
    out = b.cache.attend(**a, scale=scale, causal=False)
    assert b.cache.status() == 0
    q = _np(b.q)
    want = np.concatenate([ref.attend_all(q[x:y], k, v, b.scale if scale is None else scale)
                           for x, y, (k, v) in zip(b.offsets, b.offsets[1:], b.keys)])
    _close(out, want, b.vmax)
    assert torch.equal(out, b.cache.attend(**a, scale=scale, causal=False))
    return b, out


@pytest.mark.parametrize("D,G,page", [(64, 1, 16), (128, 4, 64), (64, 3, 32), (128, 8, 128), (128, 16, 256)])
def test_single_tokens_over_an_encoder(D, G, page):
    kv = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 129, 255, 256, 300, 1500]
    b, out = _cross(kv, [1] * len(kv), D, 2, G, page, seed=D + G)
    assert not out[0].any()


@pytest.mark.parametrize("D,G,page", [(64, 4, 16), (128, 4, 64), (128, 5, 16), (64, 40, 256)])
def test_ragged_queries_over_an_encoder(D, G, page):
    # more queries than positions and fewer; nothing to see; nothing to ask
    kv = [1, 5, 64, 65, 200, 33, 0, 7, 3, 130, 16, 0, 900]
    new = [70, 5, 200, 1, 7, 64, 0, 0, 6, 129, 33, 40, 2]
    b, out = _cross(kv, new, D, 2, G, page, seed=3)
    first = sum(new[:11])
    assert not out[first:first + 40].any()


@pytest.mark.parametrize("kv,new,G,scale", [([6000], [70], 4, None), ([300, 9000, 5, 2600], [300, 33, 5, 40], 8, -0.1),
                                            ([50000, 3], [1, 1], 4, None), ([700], [900], 1, 0.0)])
def test_long_encoders_are_cut_and_joined(kv, new, G, scale):
    _cross(kv, new, 128, 1, G, 64, seed=21, scale=scale)


def test_encoder_in_a_graph_on_a_stream():
    b, out = _cross([40, 300, 0], [50, 1, 3], 64, 2, 4, 32, seed=2)
    a = b.args()
    for k in ("group_offsets", "prefix_row", "prefix_len", "shared_len"):
        del a[k]
    got, stream, graph = torch.zeros_like(out), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    b.cache.attend(**a, out=got, stream=stream, causal=False)
    stream.synchronize()
    assert torch.equal(got, out)
    with torch.cuda.graph(graph):
        b.cache.attend(**a, out=got, causal=False)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out)


# ---------------------------------------------------------------------------------------
# forks
# ---------------------------------------------------------------------------------------

def test_forks_share_whole_pages_and_give_back_their_own():
    from segmented_rank_gemm_gb300.kv import PageTable
    page, B = 16, 6
    t = PageTable(40, page, B, 8, 200)
    t.step(_ints([70, 0, 0, 33, 0, 0]))          # 5 and 3 pages
    t.fork(_ints([-1, 0, 0, -1, 3, 0]), _ints([0, 100, 47, 0, 33, 0]))
    assert t.fork_status() == 0
    assert t.kv_len.tolist() == [70, 64, 32, 33, 32, 0] and t.shared_len.tolist() == [0, 64, 32, 0, 32, 0]
    table = t.block_table.cpu()
    assert table[1, :4].tolist() == table[0, :4].tolist() and table[2, :2].tolist() == table[0, :2].tolist()
    assert table[4, :2].tolist() == table[3, :2].tolist()
    t.step(_ints([1, 17, 1, 0, 40, 2]))
    assert t.status()[1:4] == (40 - 8 - 7, 7, 0)  # 0, 2, 1, 0, 3 and 1 pages taken
    assert t.kv_slot[1:18].tolist() == [int(t.block_table[1, (64 + i) // 16]) * 16 + i % 16 for i in range(17)]
    t.release(_ints([0, 1, 0, 0, 1, 0]))
    assert t.status()[1] == 40 - 8 - 7 + 5 and t.status()[4] == 0
    assert t.kv_len.tolist() == [71, 0, 33, 33, 0, 2] and t.shared_len.tolist() == [0, 0, 32, 0, 0, 0]
    t.release(_ints([1, 1, 1, 1, 1, 1]))
    assert t.status()[1] == 40 and sorted(t.free_pages.tolist()) == list(range(40))
    t.fork(_ints([-1, 0, -1, -1, -1, -1]))      # an empty parent: an empty child
    assert t.fork_status() == 0 and t.kv_len.tolist() == [0] * B


def test_forks_and_releases_that_cannot_be():
    from segmented_rank_gemm_gb300.kv import lora_kv_fork, lora_kv_release_shared
    from segmented_rank_gemm_gb300.lora import LoraError
    table = _ints(np.arange(12).reshape(3, 4))
    for parent, want, lens in (([3, -1, -1], None, [0, 16, 0]), ([-2, -1, -1], None, [0, 16, 0]),
                               ([1, -1, -1], None, [5, 16, 0]), ([1, 2, -1], None, [0, 0, 16]),
                               ([0, -1, -1], None, [0, 0, 0]), ([1, -1, -1], [-1, 0, 0], [0, 16, 0]),
                               ([1, -1, -1], None, [0, 65, 0]), ([1, -1, -1], None, [0, -1, 0])):
        n, s, st, tb = _ints(lens), _ints([0, 0, 0]), _ints([9]), table.clone()
        lora_kv_fork(_ints(parent), None if want is None else _ints(want), n, s, 16, tb, st)
        assert int(st) == 1 and n.tolist() == lens and s.tolist() == [0] * 3 and torch.equal(tb, table)
    free = _ints(np.zeros(9))
    for lens, shared in (([40, 0, 0], [-16, 0, 0]), ([40, 0, 0], [8, 0, 0]), ([40, 0, 0], [48, 0, 0])):
        n, s, st, top = _ints(lens), _ints(shared), _ints([9]), _ints([0])
        lora_kv_release_shared(_ints([1, 1, 1]), n, s, 16, table, free, top, st)
        assert int(st) == 1 and n.tolist() == lens and s.tolist() == shared and int(top) == 0
    with pytest.raises(LoraError):
        lora_kv_fork(_ints([0]), None, _ints([0, 0]), _ints([0, 0]), 16, table, _ints([0]))
    with pytest.raises(LoraError):
        lora_kv_release_shared(_ints([1] * 3), _ints([0] * 3), _ints([0]), 16, table, free, _ints([0]), _ints([0]))


def test_a_prompt_forked_and_continued():
    """A prompt cached once, forked into samples that then decode with the prefix shared, steps and
    maps through ``PageTable``, keys rotated on the way."""
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable, Rotary
    page, hkv, G, D, n = 16, 2, 4, 64, 9
    B, prompt = n + 1, 75
    pages = PageTable(80, page, B, 10, 128)
    cache, rotary = KvCache(80, page, hkv, D, B), Rotary(200, 32)
    gen = torch.Generator().manual_seed(3)
    held = [([], []) for _ in range(B)]
    table = rotary.angles.cpu().numpy()

    def step(new, shared):
        T = sum(new)
        q, k, v = (torch.randn(T, h, D, generator=gen).bfloat16() for h in (hkv * G, hkv, hkv))
        pages.step(_ints(new))
        qd = cache.append_rotated(q.to(DEV), k.to(DEV), v.to(DEV), pages.position[:T], pages.kv_slot[:T], rotary)
        at = [qd, pages.q_offsets, pages.kv_len, pages.block_table, max(new)]
        if shared:  # the samples, behind the prompt's own row 0
            out = cache.attend_shared(*at, _ints([1, B]), _ints([0]), _ints([64]), pages.shared_len)
        else:
            out = cache.attend(*at)
        assert cache.status() == 0 and pages.status()[3] == 0
        pos = pages.position[:T].cpu().numpy()
        cs = table[pos]
        kr = ref.held(ref.rotated(_np(k), cs[:, 0], cs[:, 1], False))
        row = 0
        for b, m in enumerate(new):
            held[b][0].extend(kr[row:row + m])
            held[b][1].extend(ref.held(_np(v))[row:row + m])
            if m:
                want = ref.attend(_np(qd)[row:row + m], np.array(held[b][0]), np.array(held[b][1]), D ** -0.5)
                _close(out[row:row + m], want, 3.5, "request %d" % b)
            row += m

    step([prompt] + [0] * n, False)
    pages.fork(_ints([-1] + [0] * n))
    for b in range(1, B):
        held[b] = ([*held[0][0][:64]], [*held[0][1][:64]])
    step([0] + [11] * n, True)  # the prompt's end and the question, in each sample
    for i in range(3):
        step([0] + [1 + (b + i) % 2 for b in range(n)], True)
    pages.release(_ints([0] + [1, 0] * (n // 2) + [1]))
    for b in range(1, B, 2):
        held[b] = ([], [])
    step([0] + [b % 2 for b in range(n)], True)
    assert pages.shared_len.tolist()[1::2] == [0] * (n // 2 + 1)
