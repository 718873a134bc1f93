"""Counts of a page's holders that are too small for the requests that end, and large forks in a graph."""
import numpy as np
import pytest
import torch

from block_sparse_long_pool_gb300 import binding
from tests.test_fork_gpu import Pool

pytestmark = pytest.mark.gpu


def twice(pool):
    pool.table[0, 1] = pool.table[0, 0]


def two(pool):
    pool.table[1, 0] = pool.table[0, 0]


def three(pool):
    pool.table[1, 0] = pool.table[2, 0] = pool.table[0, 0]
    pool.extra[pool.table[0, 0]] = 1


@pytest.mark.parametrize("max_blocks", [4, 20000])   # one CTA, a cluster
@pytest.mark.parametrize("share", [twice, two, three])
def test_a_count_that_is_too_small_is_reported(share, max_blocks):
    pool = Pool([130, 70, 5], max_blocks, 12)
    share(pool)
    pool.status.fill_(binding.SPARSE_ERR_NO_PAGES)
    pool.call([-1, -1, -1])
    torch.cuda.synchronize()
    assert pool.status.item() == binding.SPARSE_ERR_BAD_INDEX
    assert (pool.extra >= 0).all() and 0 <= int(pool.n_free) <= 12


def test_counts_end_at_zero():
    # unshared pages alone, shared ones alone, both: books as before
    pool = Pool([130, 70, 640, 0, 0], 2000, 40, seed=2)
    pool.step([0, -1, 2, 2, 0])
    pool.step([-1, 2, 2, 3, 4])
    pool.step([2, -1, 2, -1, -1])
    pool.step([-1, -1, -1, -1, -1])
    assert (pool.extra == 0).all() and int(pool.n_free) == 40


def test_a_large_fork_in_a_graph():
    B = 64
    pool = Pool([64 * 40 + 1] + [0] * (B - 1), 600, 200, seed=3)   # a cluster: its size is looked up in the capture
    t = lambda v: torch.tensor(np.asarray(v, np.int32), device="cuda")
    fork, end = t([0] * B), t([0] + [-1] * (B - 1))
    args = (pool.lens, pool.table, pool.extra, pool.free, pool.n_free, pool.copy_src, pool.copy_dst, pool.ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.sparse_page_fork(fork, *args, status=pool.status)
        binding.sparse_page_fork(end, *args, status=pool.status)
    before = sorted(pool.free[: int(pool.n_free)].tolist())
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert pool.status.item() == 0 and (pool.extra == 0).all() and pool.lens.tolist() == [64 * 40 + 1] + [0] * (B - 1)
    assert sorted(pool.free[: int(pool.n_free)].tolist()) == before
