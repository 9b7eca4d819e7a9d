"""Pages that forked requests hold stay until the last of them is released."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
HELD = 4  # include/lora_kv.h: lora_kv_release_shared


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _state(t):
    return [x.tolist() for x in (t.kv_len, t.shared_len, t.block_table, t.n_free)] + [
        t.free_pages[:int(t.n_free)].tolist()]


def test_a_parent_is_not_released_before_its_children():
    from segmented_rank_gemm_gb300.kv import PageTable
    t = PageTable(20, 16, 4, 6, 100)
    t.step(_ints([40, 0, 0, 0]))
    t.fork(_ints([-1, 0, 0, -1]))
    t.step(_ints([0, 3, 20, 5]))
    before = _state(t)
    for done in ([1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 1]):
        t.release(_ints(done))
        assert t.status()[4] == HELD and _state(t) == before, done
    t.release(_ints([0, 1, 0, 1]))          # children and strangers
    assert t.status()[4] == 0 and t.kv_len.tolist() == [40, 0, 52, 0]
    t.release(_ints([1, 0, 1, 0]))          # the parent with its last child
    assert t.status()[4] == 0 and t.kv_len.tolist() == [0] * 4
    assert sorted(t.free_pages.tolist()) == list(range(20))


def test_children_of_children():
    from segmented_rank_gemm_gb300.kv import PageTable
    t = PageTable(30, 16, 5, 6, 200)
    t.step(_ints([33, 0, 0, 0, 0]))                  # 2 whole pages
    t.fork(_ints([-1, 0, -1, -1, -1]))
    t.step(_ints([0, 40, 0, 0, 0]))                  # 72 positions, pages 2 and 3 its own
    t.fork(_ints([-1, -1, 1, 1, -1]), _ints([0, 0, 64, 32, 0]))  # 4 and 2 pages; the latter are request 0's
    assert t.fork_status() == 0 and t.shared_len.tolist() == [0, 32, 64, 32, 0]
    t.step(_ints([0, 0, 1, 1, 0]))
    before = _state(t)
    for done in ([1, 0, 0, 0, 0], [0, 1, 0, 0, 0], [1, 1, 0, 1, 0], [1, 1, 1, 0, 0]):
        t.release(_ints(done))
        assert t.status()[4] == HELD and _state(t) == before, done
    t.release(_ints([0, 1, 1, 0, 0]))  # request 3 has only pages of request 0
    assert t.status()[4] == 0
    t.release(_ints([1, 0, 0, 1, 0]))
    assert t.status()[4] == 0 and sorted(t.free_pages.tolist()) == list(range(30))


def test_a_child_that_shares_nothing_holds_nothing():
    from segmented_rank_gemm_gb300.kv import PageTable
    t = PageTable(20, 16, 3, 6, 100)
    t.step(_ints([15, 40, 0]))
    t.fork(_ints([-1, -1, 1]), _ints([0, 0, 10]))     # no whole page
    t.step(_ints([0, 0, 7]))
    t.release(_ints([0, 1, 0]))
    assert t.status()[4] == 0 and t.kv_len.tolist() == [15, 0, 7]
    # the pages given back go to others, whose rows then name them behind the table's old entries
    t.step(_ints([0, 50, 0]))
    t.release(_ints([1, 0, 1]))
    assert t.status()[4] == 0 and t.kv_len.tolist() == [0, 50, 0]


def test_many_requests():
    from segmented_rank_gemm_gb300.kv import PageTable
    rng = np.random.default_rng(1)
    B, page = 3000, 16
    t = PageTable(20000, page, B, 8, 60000)
    parents = B // 3
    t.step(_ints([int(rng.integers(16, 60)) if b < parents else 0 for b in range(B)]))
    of = [-1] * parents + [int(rng.integers(0, parents)) for _ in range(B - parents)]
    t.fork(_ints(of))
    t.step(_ints([0] * parents + [1] * (B - parents)))
    before = _state(t)
    taken = set(of[parents:])
    free = [b for b in range(parents) if b not in taken]
    held = max(taken)
    t.release(_ints([int(b in free or b == held) for b in range(B)]))
    assert t.status()[4] == HELD and _state(t) == before
    t.release(_ints([int(b in free) for b in range(B)]))
    assert t.status()[4] == 0
    t.release(_ints([int(b == held or of[b] == held) for b in range(B)]))
    assert t.status()[4] == 0
    t.release(_ints([1] * B))
    assert t.status()[4] == 0 and sorted(t.free_pages.tolist()) == list(range(20000))


def test_as_many_requests_as_there_may_be():
    from segmented_rank_gemm_gb300.kv import PageTable
    B = 16384
    t = PageTable(40, 16, B, 4, 64)
    t.step(_ints([40] + [0] * (B - 1)))
    t.fork(_ints([-1] + [0] * (B - 1)))
    assert t.fork_status() == 0 and t.shared_len.tolist() == [0] + [32] * (B - 1)
    for done, status in ([1] * (B - 1) + [0], HELD), ([0] + [1] * (B - 2) + [0], 0), ([1] + [0] * (B - 1), HELD):
        t.release(_ints(done))
        assert t.status()[4] == status and t.status()[1] == 37
    t.release(_ints([1] * B))
    assert t.status()[4] == 0 and sorted(t.free_pages.tolist()) == list(range(40))


def test_release_in_a_graph():
    from segmented_rank_gemm_gb300.kv import PageTable
    t = PageTable(20, 16, 2, 6, 100)
    t.step(_ints([40, 0]))
    t.fork(_ints([-1, 0]))
    done = _ints([1, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.release(done)
    graph.replay()
    assert t.status()[4] == HELD and t.kv_len.tolist() == [40, 32]
    done.copy_(_ints([0, 1]))
    graph.replay()
    assert t.status()[4] == 0 and t.kv_len.tolist() == [40, 0]
    done.copy_(_ints([1, 0]))
    graph.replay()
    assert t.status()[4] == 0 and sorted(t.free_pages.tolist()) == list(range(20))
