"""Queries and keys turned by their positions on the way into the 4-bit cache, on the GPU.

Tolerances.  Against the definition in fp32, whose products and sums are each rounded by itself,
everything is exact.  Against 64 bits a query is off by its rounding to bf16 (half a step, 2^-8 of
it), and by fp32's: two products, a sum and the table's rounding of a cosine of at most 1, four
halves of 2^-23 of (|a| + |b|), 2^-22 of it.
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


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16()


def _same(got, want):
    """Equal bits, but for the bits of a NaN."""
    got, want = got.cpu(), want
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


def _case(T, hq, hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(2 * torch.randn(T, 1, 1, generator=g))
    return tuple((torch.randn(T, h, D, generator=g) * size).bfloat16() for h in (hq, hkv, hkv))


def _angles(rotary, position):
    t = rotary.angles.cpu().numpy()[np.asarray(position)]
    return t[..., 0, :], t[..., 1, :]


@pytest.mark.parametrize("D,rotary", [(64, 64), (64, 32), (128, 128), (128, 96), (128, 64), (128, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,page,g", [(1, 1, 16, 1.0), (24, 3, 64, 1 / 3), (40, 8, 256, 0.02)])
def test_queries_and_cached_keys_are_exact(D, rotary, interleaved, hq, hkv, page, g):
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    T, pages, most = 77, 12, 500
    q, k, v = _case(T, hq, hkv, D, D + rotary)
    k[0], v[1] = 0, 0
    k[2], v[2] = 1e-7, 1e30
    k[3, :, 5], v[3, :, 7], q[3, 0, 1] = float("nan"), float("inf"), float("nan")
    k[4, :, 2] = float("-inf")
    k[5], k[6] = 1e-38, 3e38
    gen = torch.Generator().manual_seed(T)
    position = torch.randint(0, most, (T,), generator=gen).numpy()
    position[[7, 8]] = 0, most - 1
    slots = torch.randperm(pages * page, generator=gen)[:T].int()
    slots[10], slots[11] = -1, -1
    cache = KvCache(pages, page, hkv, D, 1, g, 2 * g)
    table = Rotary(most, rotary, interleaved=interleaved)
    out = cache.append_rotated(q.to(DEV), k.to(DEV), v.to(DEV), _ints(position), slots.to(DEV), table)
    gk, gv = cache.read(slots.to(DEV))
    assert cache.status() == 0
    cos, sin = _angles(table, position)
    assert _same(out, _bf16(ref.rotated(_np(q), cos, sin, interleaved)))
    for got, x, s in ((gk, ref.rotated(_np(k), cos, sin, interleaved), g), (gv, _np(v), 2 * g)):
        want = _bf16(ref.held(x, s))
        want[10:12] = 0
        assert torch.equal(got.cpu(), want)
    rest = torch.from_numpy(np.setdiff1d(np.arange(pages * page), slots.numpy())).int()
    rk, rv = cache.read(rest.to(DEV))
    assert not rk.any() and not rv.any()
    cache.close()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [1, 2, 333, 3000])
def test_far_positions_against_64_bits(T, interleaved):
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    D, hq, hkv, most, theta = 128, 8, 2, 1 << 18, 500000.0
    q, k, v = _case(T, hq, hkv, D, T)
    position = np.random.default_rng(T).integers(0, most, T)
    position[0] = most - 1
    cache = KvCache(T // 64 + 1, 64, hkv, D, 1)
    table = Rotary(most, D, theta, interleaved)
    out = cache.append_rotated(q.to(DEV), k.to(DEV), v.to(DEV), _ints(position), _ints(np.arange(T)), table)
    angle = position[:, None] * np.power(theta, -np.arange(0, D, 2) / D)
    want = ref.rotated(_np(q), np.cos(angle), np.sin(angle), interleaved, np.float64)
    x = np.abs(_np(q).astype(np.float64))
    pair = np.concatenate((x[..., 64:], x[..., :64]), -1) if not interleaved else x.reshape(
        T, hq, 64, 2)[..., ::-1].reshape(T, hq, D)
    lim = 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * (x + pair)
    assert (np.abs(_np(out).astype(np.float64) - want) <= lim).all()
    assert cache.status() == 0
    cache.close()


def test_position_zero_is_append():
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    T, hq, hkv, D = 100, 4, 2, 64
    q, k, v = (x.to(DEV) for x in _case(T, hq, hkv, D, 5))
    a, b = KvCache(8, 16, hkv, D, 1), KvCache(8, 16, hkv, D, 1)
    slots = _ints(np.random.default_rng(0).permutation(128)[:T])
    a.append(k, v, slots)
    out = b.append_rotated(q, k, v, _ints(np.zeros(T)), slots, Rotary(1, 32))
    assert torch.equal(out, q)
    for x, y in zip(a.read(slots), b.read(slots)):
        assert torch.equal(x, y)


def test_packed_rows_in_place_on_a_stream_and_in_a_graph():
    # q, k and v as columns of one projection's rows, q turned where it is
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    T, hq, hkv, D = 70, 6, 2, 128
    q, k, v = _case(T, hq, hkv, D, 9)
    position = np.arange(T) * 3
    table = Rotary(300, 96)
    want = _bf16(ref.rotated(_np(q), *_angles(table, position), False))
    rows = torch.cat((q.flatten(1), k.flatten(1), v.flatten(1)), 1)
    slots = _ints(np.arange(T))
    pos = _ints(position)

    def parts(x):
        return (x[:, :hq * D].view(T, hq, D), x[:, hq * D:(hq + hkv) * D].view(T, hkv, D),
                x[:, (hq + hkv) * D:].view(T, hkv, D))

    cache = KvCache(8, 16, hkv, D, 1)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    buf = rows.to(DEV)
    qd, kd, vd = parts(buf)
    torch.cuda.synchronize()
    out = cache.append_rotated(qd, kd, vd, pos, slots, table, q_out=qd, stream=stream)
    stream.synchronize()
    assert out.data_ptr() == qd.data_ptr() and torch.equal(out.cpu(), want)
    assert torch.equal(buf[:, hq * D:].cpu(), rows[:, hq * D:])
    held = cache.read(slots)
    buf.copy_(rows)
    torch.cuda.synchronize()
    other = KvCache(8, 16, hkv, D, 1)
    with torch.cuda.graph(graph):
        other.append_rotated(qd, kd, vd, pos, slots, table, q_out=qd)
    for _ in range(2):
        buf.copy_(rows)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qd.cpu(), want)
    for x, y in zip(held, other.read(slots)):
        assert torch.equal(x, y)


def test_positions_and_slots_that_only_the_call_holds():
    # tensors made in the call's expression stay until it has been made: an output that the call
    # allocates is not their memory
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    q, k, v = _case(1, 8, 2, 128, 1)
    table, cache = Rotary(1000, 128), KvCache(1, 64, 2, 128, 1)
    want = _bf16(ref.rotated(_np(q), *_angles(table, [999]), False))
    for _ in range(20):
        torch.cuda.empty_cache()
        out = cache.append_rotated(q.to(DEV), k.to(DEV), v.to(DEV), _ints([999]), _ints([5]), table)
        assert cache.status() == 0 and torch.equal(out.cpu(), want)
    cache.close()


def test_positions_and_slots_outside_are_flagged_and_left_alone():
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    from segmented_rank_gemm_gb300.lora import LORA_EID
    T, hq, hkv, D = 8, 4, 2, 64
    q, k, v = _case(T, hq, hkv, D, 3)
    table = Rotary(10, 64)
    good_pos, good_slot = np.arange(T), np.arange(T) * 2
    for pos, slot in (({2: -1}, {}), ({3: 10}, {}), ({4: 2 ** 31 - 1}, {}), ({}, {5: 32}), ({}, {5: -2})):
        cache = KvCache(2, 16, hkv, D, 1)
        position, slots = good_pos.copy(), good_slot.copy()
        for b, x in pos.items():
            position[b] = x
        for b, x in slot.items():
            slots[b] = x
        out = torch.full_like(q, 7.0, device=DEV)
        cache.append_rotated(q.to(DEV), k.to(DEV), v.to(DEV), _ints(position), _ints(slots), table, q_out=out)
        assert cache.status() == LORA_EID and cache.status() == 0
        want = _bf16(ref.rotated(_np(q), *_angles(table, good_pos), False))
        for b in pos:
            want[b] = 7.0
        assert torch.equal(out.cpu(), want)
        gk, gv = cache.read(_ints(good_slot))
        wk = _bf16(ref.held(ref.rotated(_np(k), *_angles(table, good_pos), False)))
        wv = _bf16(ref.held(_np(v)))
        for b in list(pos) + list(slot):
            wk[b], wv[b] = 0, 0
        assert torch.equal(gk.cpu(), wk) and torch.equal(gv.cpu(), wv)
        cache.close()


def test_refusals():
    from segmented_rank_gemm_gb300.kv import KvCache, Rotary
    from segmented_rank_gemm_gb300.lora import LoraError
    for args in ((0, 64), (4, 16), (4, 48), (4, 0)):
        with pytest.raises(ValueError):
            Rotary(*args)
    with pytest.raises(ValueError):
        Rotary(4, 64, frequencies=torch.ones(16))
    T, hq, hkv, D = 3, 4, 2, 64
    cache = KvCache(2, 16, hkv, D, 1)
    q, k, v = (x.to(DEV) for x in _case(T, hq, hkv, D, 3))
    rows = torch.zeros(T, (hq + 2 * hkv) * D, dtype=torch.bfloat16, device=DEV)
    flat = torch.zeros(2 * T * hq * D, dtype=torch.bfloat16, device=DEV)
    ok = dict(q=q, k=k, v=v, position=_ints([0, 1, 2]), kv_slot=_ints([0, 1, 2]), rotary=Rotary(4, 64))
    wide, other = Rotary(4, 96), Rotary(4, 64, device="cpu")
    with pytest.raises(AttributeError):
        other.angles = other.angles[:3]
    shifted = flat[8:8 + T * hq * D].view(T, hq, D)
    for change in (dict(q=q.float()), dict(k=k[:2]), dict(v=v.float()), dict(position=_ints([0, 1])),
                   dict(kv_slot=_ints([0, 1, 2]).long()), dict(rotary=wide), dict(rotary=other),
                   dict(q_out=q[:2]), dict(q=flat[:T * hq * D].view(T, hq, D), q_out=shifted),
                   dict(q_out=rows[:, :hq * D].view(T, hq, D), k=rows[:, (hq - 1) * D:(hq + 1) * D].view(T, hkv, D)),
                   dict(q_out=k.repeat(1, 2, 1)[:, :3].expand(T, 3, D)), dict(q=q.cpu())):
        with pytest.raises(LoraError):
            cache.append_rotated(**{**ok, **change})
    assert cache.status() == 0
    cache.append_rotated(**ok)
    cache.append_rotated(**{**ok, "q": q[:0], "k": k[:0], "v": v[:0], "position": ok["position"][:0],
                            "kv_slot": ok["kv_slot"][:0]})
    cache.close()
