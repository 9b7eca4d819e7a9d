"""Requests as long as a cache may be: 2^31 - 16 positions, whose tiles' last positions, counted from a page
behind the first, pass 2^31.

All keys are zeros but at a few positions, whose scores of 40 leave the others, e^40 times smaller and fewer
than 2^31, below 2^-26 of the sum: the result is the mean of the values there.  Tolerance: one rounding of
the output (2^-8), probabilities rounded to fp16 (2^-11 max|v|).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16
PAGE, D, G = 16, 64, 2
PAGES = 2 ** 27 - 1
KV = PAGES * PAGE


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def test_requests_of_two_to_the_31_positions():
    from oracle import kv as ref
    from segmented_rank_gemm_gb300.kv import KvCache
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 175e9:
        pytest.skip("needs 160 GB of device memory")
    cache = KvCache(PAGES, PAGE, 1, D, 2)
    try:
        table = torch.arange(PAGES, dtype=torch.int32, device=DEV).repeat(2, 1)
        gen = torch.Generator().manual_seed(1)
        special = [0, 15, 16, 47, 2 ** 30 + 5, KV - 65, KV - 33, KV - 17, KV - 2, KV - 1]
        k, v = torch.zeros(len(special), 1, D), torch.randn(len(special), 1, D, generator=gen)
        k[:, :, 0] = 8.0
        cache.append(k.to(BF16).to(DEV), v.to(BF16).to(DEV), _ints(special))
        held = ref.held(v.to(BF16).float().numpy())[:, 0]
        for rows in (3, 70):  # of a request: the kernel for few rows, and the one for many
            q = torch.zeros(2 * rows, G, D, dtype=BF16)
            q[:, :, 0] = 40.0
            q, at = q.to(DEV), (_ints([0, rows, 2 * rows]), _ints([KV, KV]), table, rows)
            want = np.array([held[[s < KV - rows + 1 + i for s in special]].mean(0) for i in range(rows)] * 2)
            shares = [_ints([0, 2]), _ints([0])]
            for name, out, expect in (
                    ("causal", cache.attend(q, *at), want),
                    ("shared", cache.attend_shared(q, *at, *shares, _ints([PAGE]), _ints([PAGE] * 2)), want),
                    ("long prefix", cache.attend_shared(q, *at, *shares, _ints([KV - 80]), _ints([KV - 80] * 2)), want),
                    ("cross", cache.attend(q, *at, causal=False), np.broadcast_to(held.mean(0), want.shape))):
                assert cache.status() == 0, name
                err = np.abs(out.float().cpu().numpy() - expect[:, None])
                lim = 2.0 ** -8 * np.abs(expect) + 2.0 ** -10 * np.abs(held).max()
                assert (err <= lim[:, None]).all(), (name, rows, err.max())
    finally:
        cache.close()
        del table
        torch.cuda.empty_cache()
