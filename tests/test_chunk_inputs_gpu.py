"""Chunk attention of inputs that are not as they should be: what is reported, and what stays as it was."""
import pytest
import torch

from block_sparse_long_pool_gb300 import binding
from tests.chunk_utils import Chunk

pytestmark = pytest.mark.gpu


def ws(c):
    return binding.paged_chunk_workspace(c.B, c.H_q, c.H_kv)


@pytest.mark.parametrize("cu", [[0, 40, 10, 50], [30, 30, 0, 80], [0, 40, 80, 79]])
def test_rows_of_two_requests_are_refused(cu):
    c = Chunk([100, 100, 100], [40, 0, 40], 1, 4, seed=41)
    c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    c.call(ws(c))
    torch.cuda.synchronize()
    assert c.status.item() == binding.SPARSE_ERR_BAD_INDEX
    assert (c.O == 7).all() and (c.lse == 7).all()


def test_a_bad_page_is_reported_where_the_plan_refused_a_request():
    c = Chunk([300, 50], [40, 6], 1, 4, seed=42)
    c.table[0, 2] = c.n_pages
    c.status.fill_(binding.SPARSE_ERR_NO_PAGES)
    c.call(ws(c))
    c.check(status=binding.SPARSE_ERR_BAD_INDEX)
    c.table[0, 2] = 0
    c.status.fill_(binding.SPARSE_ERR_NO_PAGES)
    c.call(ws(c))
    c.check(status=binding.SPARSE_ERR_NO_PAGES)   # a sound call leaves the word as it is
    c.table[0, 2] = c.n_pages
    c.status.fill_(binding.SPARSE_ERR_TIMEOUT)
    c.call(ws(c))
    c.check(status=binding.SPARSE_ERR_TIMEOUT)


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("start,new,row", [([70], [60], 3), ([12000], [5], 3), ([70, 30] * 90, [3, 60] * 90, 61)])
def test_infinite_queries(start, new, row, value):
    # an item of one CTA, one that many share, one of many
    c = Chunk(start, new, 1, 4, seed=43)
    w = ws(c)
    c.call(w)
    c.check()
    O, lse = c.O.clone(), c.lse.clone()
    c.Q[row, 1, 5] = value
    c.Q[row, 2, 127], c.Q[row, 2, 0] = value, -value
    c.call(w)
    torch.cuda.synchronize()
    rest = torch.ones_like(lse, dtype=torch.bool)
    rest[row, 1] = rest[row, 2] = False
    assert c.O[~rest].isnan().all() and c.lse[~rest].isnan().all()
    assert torch.equal(c.O[rest], O[rest]) and torch.equal(c.lse[rest], lse[rest])
