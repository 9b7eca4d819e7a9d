"""The plain definitions of ``oracle.kv`` pinned to closed forms and to torch, on the CPU."""
import numpy as np
import torch

from oracle import kv as ref


def test_e4m3_values_and_rounding_equal_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(codes, ref.E4M3)
    x = np.concatenate((np.random.default_rng(0).random(20000) * 500, ref.E4M3,
                        (ref.E4M3[1:] + ref.E4M3[:-1]) / 2)).astype(np.float32)
    want = torch.from_numpy(np.minimum(x, 448)).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.to_e4m3(x), want)


def test_held_values():
    x = np.zeros((1, 32), np.float32)
    x[0, :16] = np.arange(16) - 8.0   # max 8: s = e4m3(8/7) = 1.125, codes round(x / 1.125)
    got = ref.held(x)[0]
    assert got[0] == -7 * 1.125 and got[8] == 0 and got[15] == 6 * 1.125
    assert not got[16:].any()
    # The error: half a step, or, where rounding took the scale below max / 7 (by at most 1/16 of
    # it), the rest of a value beyond 7 steps.
    x = np.random.default_rng(1).standard_normal((50, 4, 64)).astype(np.float32)
    grp = x.reshape(50, 4, 4, 16)
    s = ref.to_e4m3(np.abs(grp).max(-1) / 7)[..., None]
    err = np.abs(ref.held(x).reshape(grp.shape) - grp)
    assert (err <= np.maximum(s / 2, np.abs(grp) - 7 * s) * (1 + 1e-6)).all()
    h = ref.held(x)
    assert not ref.held(h * 0).any()
    assert not ref.held(np.full((1, 16), np.nan)).any()
    assert np.array_equal(ref.held(np.array([[np.inf] + [0.0] * 15])), [[7 * 448.0] + [0.0] * 15])


def test_attend_equals_torchs_softmax():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    got = ref.attend(q, k, v, 0.3)
    tq, tk, tv = (torch.from_numpy(x) for x in (q, k, v))
    for h in range(4):
        s = 0.3 * tq[:, h] @ tk[:, h // 2].T
        hidden = torch.ones(5, 9, dtype=torch.bool).triu(9 - 5 + 1)
        want = torch.softmax(s.masked_fill(hidden, float("-inf")), -1) @ tv[:, h // 2]
        assert np.allclose(got[:, h], want.numpy(), rtol=1e-12, atol=1e-14)
    assert not ref.attend(q, k[:2], v[:2], 0.3)[:3].any()


def test_maps_by_hand():
    table = np.full((3, 3), -1, np.int32)
    table[0, 0], table[2, 0] = 7, 4
    out = ref.maps([3, 0, 4], [2, 3, 1], [5, -1, 6], 4, table, [0, 1, 2, 3], 4, 8)
    # request 0: position 3 on page 7, position 4 on a new page (3); request 1: page 2;
    # request 2: length 4 fills page 4, position 4 on page 1
    assert out["table"].tolist() == [[7, 3, -1], [2, -1, -1], [4, 1, -1]]
    assert out["kv_slot"] == [31, 12, 8, 9, 10, 4, -1, -1]
    assert out["position"] == [3, 4, 0, 1, 2, 4, 0, 0]
    assert out["token_slot"] == [5, 5, -1, -1, -1, 6, -1, -1]
    assert out["q_offsets"] == [0, 2, 5, 6] and out["kv_len"] == [5, 3, 5]
    assert out["counts"] == [6, 1, 3, 0, 0]


def test_norm_by_hand():
    h, y, s = ref.rms_norm([[3.0, 4.0]], [[0.0, 0.0]], [1.0, 2.0], 0.0)
    r = np.sqrt(12.5)
    assert np.allclose(y, [[3 / r, 8 / r]]) and np.allclose(s, [8 / r / 448])


def test_library_refuses_null_and_bad_sizes_without_a_device():
    from segmented_rank_gemm_gb300 import build
    build.build()
    import ctypes
    from segmented_rank_gemm_gb300 import lora
    L = lora.library()
    h = ctypes.c_void_p()
    assert L.lora_kv_cache_create(None, 4, 16, 1, 64, 1, 1.0, 1.0, None) == lora.LORA_EINVAL
    for args in ((0, 16, 1, 64, 1, 1.0, 1.0), (4, 17, 1, 64, 1, 1.0, 1.0), (4, 16, 257, 64, 1, 1.0, 1.0),
                 (4, 16, 1, 65, 1, 1.0, 1.0), (4, 16, 1, 64, 16385, 1.0, 1.0),
                 (4, 16, 1, 64, 1, -1.0, 1.0), (4, 16, 1, 64, 1, 1.0, float("nan"))):
        assert L.lora_kv_cache_create(ctypes.byref(h), *args, None) == lora.LORA_EINVAL
        assert not h.value
    assert L.lora_kv_append(None, 16, 64, 16, 64, 16, 1, None) == lora.LORA_EINVAL
    assert L.lora_kv_read(None, 16, 1, 16, 16, None) == lora.LORA_EINVAL
    assert L.lora_kv_attend(None, 16, 64, 1, 16, 16, 16, 1, 1, 1, 1, 1.0, 16, 64, None) == lora.LORA_EINVAL
    assert L.lora_kv_get_status(None, None) == lora.LORA_EINVAL
    assert L.lora_kv_cache_bytes(None) == 0
    L.lora_kv_cache_destroy(None)
    d = 1 << 20  # never dereferenced: validation fails first
    for B, T, page, blocks, pages in ((0, 1, 16, 1, 1), (16385, 1, 16, 1, 1), (1, -1, 16, 1, 1),
                                      (1, 1, 48, 1, 1), (1, 1, 16, 0, 1), (1, 1, 16, 1, 0),
                                      (1, 1, 256, 1 << 23, 1), (2, 1, 16, 1 << 30, 1)):
        assert L.lora_kv_maps(d, d, d, B, T, page, d, blocks, d, pages, d, d, d, d, d, d, d,
                              None) == lora.LORA_EINVAL
    assert L.lora_kv_maps(None, d, d, 1, 1, 16, d, 1, d, 1, d, d, d, d, d, d, d, None) == lora.LORA_EINVAL
    assert L.lora_kv_release(d, d, 1, 16, d, 1, d, 1, d, None, None) == lora.LORA_EINVAL
    n = lora.LORA_BF16
    bad = [(d, 7, None, 0, d, 1e-6, 1, 8, n, None, 0, d, None, None),    # ldx < K
           (d, 8, d, 7, d, 1e-6, 1, 8, n, None, 0, d, None, None),       # ldr < K
           (d, 8, None, 0, d, -1.0, 1, 8, n, None, 0, d, None, None),    # eps
           (d, 8, None, 0, d, 1e-6, 1, 8, 5, None, 0, d, None, None),    # dtype
           (d, 8, None, 0, d, 1e-6, 1, 8, n, None, 0, None, None, None),  # no output
           (d, 8, None, 0, d, 1e-6, 1, 8, n, None, 0, None, d, None),    # xq without sx
           (d, 8, None, 0, None, 1e-6, 1, 8, n, None, 0, 2 * d, None, None),
           (d, 40000, None, 0, d, 1e-6, 1, 40000, n, None, 0, d, None, None),
           (d, 8, None, 0, 2 * d, 1e-6, 4, 8, n, None, 0, d + 16, None, None)]  # y over x
    for a in bad:
        assert L.lora_rms_norm(*a, None) == lora.LORA_EINVAL, a
