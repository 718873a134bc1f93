"""The paged 8-bit cache at the ends of what it accepts: the largest table, scales far apart or
no powers of two, what the status word says, and workspaces whose call gave up."""
import numpy as np
import pytest
import torch

import paged_utils as ref
from block_sparse_long_pool_gb300 import binding
from test_paged_gpu import BLK, DEV, Plan, i32

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- page plan


@pytest.mark.parametrize("n_tok", [130, 2000])
def test_plan_of_the_largest_table(n_tok):
    """2^25 - 1 blocks: a request that fills its last one (in one launch and, with its outputs in
    place, in two), and one token more, which does not fit."""
    max_blocks = 2 ** 25 - 1
    cap = max_blocks * BLK
    s = Plan([cap - n_tok], np.zeros((1, 1)), np.arange(64)[::-1].copy(), 64, n_tok)
    s.table = torch.zeros((1, max_blocks), dtype=torch.int32, device=DEV)
    used = ref.nblk(cap - n_tok)
    s.table[0, used - 1] = 63
    pos = np.arange(cap - n_tok, cap)
    page = np.where(pos // BLK < used, 63, pos // BLK - used)   # pages 0, 1, ... from the list's end
    keep = s.table.clone()
    for in_place in (False, True):
        for add in (n_tok + 1, n_tok):
            s.n_new.fill_(add)
            s.call(in_place)
            torch.cuda.synchronize()
            if add > n_tok:
                assert s.start.tolist() == [-1] and (s.slot == -1).all()
                assert (s.seq_len if in_place else s.len_out).tolist() == [cap - n_tok]
                assert s.status.item() == binding.SPARSE_ERR_NO_PAGES and torch.equal(s.table, keep)
                s.status.zero_()
        assert s.start.tolist() == [cap - n_tok] and s.status.item() == 0
        assert (s.seq_len if in_place else s.len_out).tolist() == [cap]
        assert (s.n_free if in_place else s.n_free_out).tolist() == [64 - (max_blocks - used)]
        assert np.array_equal(s.pos.cpu().numpy(), pos) and np.array_equal(s.slot.cpu().numpy(), page * BLK + pos % BLK)
        assert torch.equal(s.table[0, used:], i32(np.arange(max_blocks - used)))
        s.table.copy_(keep)
