"""Attention of shared prefixes in the kernels that share and join, whatever the batch's size: a table as
wide as a long request's keeps small batches from being attended alone.  Every call here is seen to have
gone that way by its workspace, which a batch attended alone leaves as it was.

Tolerances: those of tests/test_shared_gpu.py.
"""
import numpy as np
import pytest
import torch

from test_shared_gpu import Batch, _close, _ints, _np

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16
MARK = 0xA5  # the workspace's bytes before a call
WIDE = 1 << 20  # positions that a request may have, by the table's width


class Sharing(Batch):
    ws = None

    def args(self, **change):
        a = super().args(**change)
        more = WIDE // self.page - a["block_table"].shape[1]
        if more > 0:  # (entries that are not read)
            a["block_table"] = torch.nn.functional.pad(a["block_table"], (0, more), value=2 ** 30).contiguous()
        if "workspace" not in change:
            q = a["q"]
            self.ws = a["workspace"] = self.cache.shared_workspace(q.shape[0], q.shape[1])
            self.ws.fill_(MARK)
        return a

    def attend(self, **change):
        out = super().attend(**change)
        assert shared(self.ws)
        return out


def shared(ws):
    return bool((ws != MARK).any())


def cut_whole_requests(ws, rows, D):
    """Which of `rows` (rows times heads) were left in pieces that are all of the row's result: a sum of
    -2 stands for that (it follows the results of both parts)."""
    n = rows
    ml = ws.view(torch.float32)[2 * n * D:2 * n * D + 2 * n].view(n, 2)
    return ml[:, 1] == -2


@pytest.mark.parametrize("D,G,page", [(64, 1, 16), (128, 4, 64), (64, 3, 32), (128, 8, 16), (128, 5, 128),
                                      (64, 11, 256)])
def test_single_tokens(D, G, page):
    rng = np.random.default_rng(D + G)
    groups = [(page, [(1, 1), (2, 1)]), (3 * page, [(n, 1) for n in (1, 15, 16, 17, 31, 33, 64, 65, 100)]),
              (7 * page, [(40, 1)]), (20 * page, [(int(rng.integers(1, 90)), 1) for _ in range(70)])]
    Sharing(groups, D, 2, G, page, seed=G).check()


@pytest.mark.parametrize("leader", [False, True])
def test_several_tokens_idle_members_and_requests_by_themselves(leader):
    groups = [(32, [(3, 3), (9, 1)]), (0, [(5, 2), (70, 1)]), (80, [(4, 0), (0, 0)]), (64, [(9, 2), (33, 5), (7, 1)])]
    Sharing(groups, 64, 1, 2, 16, seed=3, leader=leader, alone=(1, 8), outside=[(20, 2), (0, 0), (300, 1)]).check()


@pytest.mark.parametrize("prefix,members,G", [(20000, 3, 4), (9008, 2, 1), (3008, 6, 4), (16, 2, 5)])
def test_long_prefixes_of_few_rows(prefix, members, G):
    # (the kernel for few rows cuts them, and joins their pieces by itself)
    rng = np.random.default_rng(prefix)
    groups = [(prefix, [(int(rng.integers(1, 60)), 1) for _ in range(members)])]
    Sharing(groups, 128, 1, G, 16, seed=8, spread=1.4).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("members,G", [(3, 4), (40, 4), (2, 1), (70, 5)])
@pytest.mark.parametrize("far", ["prefix", "own", "both"])
def test_scores_far_apart_between_prefix_and_own_positions(far, members, G, D):
    # all of the weight in the prefix, all of it behind, and either by the token: scores of the prefix's
    # positions are some 170 powers of two above or below those behind
    rng = np.random.default_rng(members)
    b = Sharing([(320, [(int(n), int(min(n, 1 + i % 2))) for i, n in enumerate(rng.integers(1, 70, members))])],
                D, 1, G, 16, seed=11)
    k, v = (torch.randn(sum(x.shape[0] for x, _ in b.keys), 1, D, generator=torch.Generator().manual_seed(i))
            for i in (1, 2))
    # keys anew: dimension 0 tells prefix from own positions
    from oracle import kv as ref
    page, row = b.page, 0
    first = True
    for r, (kk, vv) in enumerate(b.keys):
        n = kk.shape[0]
        where = [int(b.table[r, p // page]) * page + p % page for p in range(n)]
        x, y = k[row:row + n].clone(), v[row:row + n]
        if not first:  # the prefix's keys are one and the same
            x[:320], y[:320] = k[:320], v[:320]
        x[:320, :, :16], x[320:, :, :16] = 0, 0
        x[:320, :, 0], x[320:, :, 0] = 6.0, -6.0
        b.cache.append(x.to(BF16).to(DEV), y.to(BF16).to(DEV), _ints(where))
        b.keys[r] = (ref.held(_np(x.to(BF16))), ref.held(_np(y.to(BF16))))
        row, first = row + n, False
    b.vmax = max(np.abs(y).max() for _, y in b.keys)
    sign = {"prefix": 1.0, "own": -1.0}.get(far)
    b.q[:, :, 1:16] = 0
    rows = torch.arange(b.q.shape[0]) % 2 * 2.0 - 1
    b.q[:, :, 0] = (rows if sign is None else torch.full_like(rows, sign))[:, None] * 10 * D ** 0.5
    out = b.attend()
    assert b.cache.status() == 0
    _close(out, b.expected(), b.vmax)


def test_nan_queries_stay_in_their_rows():
    b = Sharing([(64, [(10, 1), (20, 1), (30, 12)])], 128, 2, 4, 16, seed=12)
    want, bad = b.expected(), b.q.clone()
    bad[1, 2, 17] = float("nan")
    out = _np(b.attend(q=bad.to(DEV)))
    assert np.isnan(out[1, 2]).all()
    mask = np.ones(out.shape[:2], bool)
    mask[1, 2] = False
    _close(torch.from_numpy(out[mask]), want[mask], b.vmax)


@pytest.mark.parametrize("groups", [[(256, [(10, 1), (20, 3), (30, 1)]), (64, [(5, 1)] * 9)],
                                    [(256, [(10, 2)] * 40), (64, [(90, 70), (5, 1)])]])
def test_strided_rows_padding_streams_and_a_graph(groups):
    b = Sharing(groups, 64, 2, 4, 64, seed=13)
    want, T, width = b.expected(), sum(b.new), 8 * 64
    wide = torch.full((T + 5, width + 64), 9.0, dtype=BF16, device=DEV)
    q = wide[:, 8:8 + width].view(T + 5, 8, 64)
    q[:T] = b.q.to(DEV)
    outw = torch.full((T + 5, width + 8), 5.0, dtype=BF16, device=DEV)
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
    assert not ws.view(torch.float32).isnan().all()
    once = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.cache.attend_shared(**a)
    for _ in range(3):
        out.fill_(3.0)
        ws.view(torch.float32).fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, once) and not ws.view(torch.float32).isnan().all()


def test_calls_without_a_pause_share_a_workspace():
    # prefixes of many rows and of few in turn, each call reading what the one before wrote
    a = Sharing([(2048, [(20, 1)] * 40)], 128, 2, 4, 64, seed=14)
    b = Sharing([(512, [(7, 1)] * 2), (64, [(100, 1)] * 3)], 128, 2, 4, 64, seed=15)
    ws = torch.empty(a.cache.shared_workspace(40, 8).numel(), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(x.q, device=DEV) for x in (a, b)]
    args = [x.args(out=o, workspace=ws) for x, o in zip((a, b), outs)]
    for x, k in zip((a, b), args):
        ws.fill_(MARK)
        x.cache.attend_shared(**k)
        assert shared(ws)
    for _ in range(20):
        for x, k in zip((a, b), args):
            x.cache.attend_shared(**k)
    for x, o in zip((a, b), outs):
        _close(o, x.expected(), x.vmax)
        assert x.cache.status() == 0


def test_two_at_a_time():
    parts = []
    for seed in (11, 12):
        b = Sharing([(480 + 16 * seed, [(9 + i, 1 + i % 3) for i in range(4 + 40 * (seed - 11))]),
                     (64, [(300, 200)])], 128, 2, 4, 16, seed=seed, outside=[(500, 120)])
        a = b.args(out=torch.empty_like(b.q, device=DEV))
        parts.append((b, a, torch.cuda.Stream()))
    want = []
    torch.cuda.synchronize()
    for b, a, stream in parts:
        b.cache.attend_shared(**a, stream=stream)
        torch.cuda.synchronize()
        assert shared(a["workspace"])
        _close(a["out"], b.expected(), b.vmax)
        want.append(a["out"].clone())
    torch.cuda.synchronize()
    for _ in range(30):
        for b, a, stream in parts:
            b.cache.attend_shared(**a, stream=stream)
        torch.cuda.synchronize()
        for (b, a, _), w in zip(parts, want):
            assert torch.equal(a["out"], w)
    assert all(b.cache.status() == 0 for b, _, _ in parts)


def test_what_cannot_be_is_flagged():
    from segmented_rank_gemm_gb300.lora import LORA_EID
    b = Sharing([(64, [(20, 1), (30, 2)]), (128, [(9, 1), (40, 1)])], 64, 1, 4, 32, seed=16)
    want, shared_len, extra = b.expected(), list(b.shared), [0, 0]
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
    assert b.cache.status() == 0 and b.shared == shared_len
    b.check()


@pytest.mark.parametrize("G,D", [(4, 128), (3, 64), (5, 128)])
@pytest.mark.parametrize("where", ["only", "member", "outside"])
def test_requests_without_a_prefix_that_are_cut(where, G, D):
    # more than 256 rows a head over thousands of positions: cut between CTAs, and all of its rows' result
    long = (5000, 300)
    if where == "only":
        b = Sharing([(64, [long])], D, 1, G, 16, seed=G, alone=(0,))
    elif where == "member":
        b = Sharing([(640, [(30, 1), (5000 - 640, 300), (7, 2)])], D, 1, G, 16, seed=G, alone=(1,))
    else:
        b = Sharing([(640, [(30, 1), (64, 30), (7, 2)])], D, 1, G, 16, seed=G, outside=[long])
    b.check()
    row = 0 if where == "only" else 1 if where == "member" else 33
    cut = cut_whole_requests(b.ws, b.q.shape[0] * G, D).view(-1, G)
    assert cut[row:row + 300].any() and not cut[:row].any() and not cut[row + 300:].any()


def test_prompts_that_share_nothing_beside_tokens_that_share():
    b = Sharing([(512, [(1 + 3 * i, 1) for i in range(60)]), (0, [(200, 200)])], 128, 2, 4, 64, seed=5,
                outside=[(448, 448), (700, 64), (33, 33)])
    b.check()


@pytest.mark.parametrize("many", [False, True])
def test_a_block_on_a_wide_page_table(many):
    """A forked prompt through a block in a graph and on a stream, on a table as wide as its longest request
    may get, with the samples' prefix shared."""
    from segmented_rank_gemm_gb300.kv import KvCache, PageTable, Rotary
    from test_decoder_gpu import D, HIDDEN, KV, _attention, _mlp, _rows
    B, page = (60 if many else 5), 16
    T = 4 * B
    cache, pages, rotary = KvCache(400, page, KV, D, B), PageTable(400, page, B, WIDE // page, T), Rotary(400, 64)
    block, (mlp, _) = _attention(T, cache, rotary=rotary, share=True), _mlp(T)
    alone = _attention(T, cache, rotary=rotary)
    prompt = min(T, 200)
    shared_len = prompt // page * page
    n = torch.zeros(B, dtype=torch.int32)
    n[0] = prompt
    pages.step(n.to(DEV), _ints([1] * B))
    block.forward(_rows(prompt, 1), _rows(prompt, 2), pages, prompt)
    pages.fork(_ints([-1] + [0] * (B - 1)))
    torch.cuda.synchronize()
    state = {k: getattr(pages, k).clone() for k in ("kv_len", "block_table", "counts", "shared_len")}
    groups = (_ints([1, B]), _ints([0]), _ints([shared_len]))
    new, ids, rows = _ints([0] + [2] * (B - 1)), _ints([1] * B), 2 * (B - 1)
    x, h, y = _rows(rows, 3), _rows(rows, 4), torch.empty(rows, HIDDEN, dtype=BF16, device=DEV)
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
        block.parts.fill_(MARK)
        torch.cuda.synchronize()

    reset()
    step()
    torch.cuda.synchronize()
    assert shared(block.parts)
    want, ctx = h.clone(), block.ctx[:rows].clone()
    reset()
    pages.step(new, ids)
    alone.forward(x, h.clone(), pages, 2)
    torch.cuda.synchronize()
    assert not shared(block.parts)
    # the same sums in another order: both within their tolerance of the definition
    vmax = cache.read(torch.arange(400 * page, dtype=torch.int32, device=DEV))[1].float().abs().max()
    err = (alone.ctx[:rows].float() - ctx.float()).abs()
    assert (err <= 2.0 ** -7 * ctx.float().abs() + 2.0 ** -9 * vmax).all()
    reset()
    stream = torch.cuda.Stream()
    step(stream)
    stream.synchronize()
    assert torch.equal(h, want) and shared(block.parts)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want) and shared(block.parts)
    assert cache.status() == 0 and pages.status()[3] == 0
