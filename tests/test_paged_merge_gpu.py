"""Decode attention over the paged 8-bit cache where a pair's tiles lie in many CTAs: every
listed block counts once, whatever its place, and every merge reads its own call's states."""
import numpy as np
import pytest
import torch

from block_sparse_long_pool_gb300 import binding
from test_paged_gpu import BLK, D, DEV, F8, Attn, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,G,blocks", [(1, 1, 1, 700), (1, 2, 4, 300), (2, 4, 8, 160), (1, 1, 16, 2048), (5, 3, 9, 77)])
def test_merges_read_the_states_of_their_own_call(B, H, G, blocks):
    """Calls queued one behind another on one workspace, each over pages of another constant: with
    queries of zero all weights are 1, so that O is that constant, once rounded to bf16, unless a
    state of the call before was merged."""
    consts = [1.0, -3.0, 0.5, 24.0, -0.0625]
    pages = torch.empty((len(consts), H, 2, BLK, D), device=DEV)
    for i, x in enumerate(consts):
        pages[i] = x
    pages = pages.to(F8)
    scale = torch.ones((len(consts), H, 2), device=DEV)
    Q = torch.zeros((B, H * G, D), dtype=torch.bfloat16, device=DEV)
    tables = [torch.full((B, blocks), i, dtype=torch.int32, device=DEV) for i in range(len(consts))]
    lens = i32([blocks * BLK - b for b in range(B)])
    a = Attn(B, H * G, H)
    got = []
    for n in range(100):
        O = torch.full((B, H * G, D), 7.0, dtype=torch.bfloat16, device=DEV)
        binding.sparse_paged_decode_attn_f8(Q, pages, scale, tables[n % len(consts)], lens, O, a.ws, lse=a.lse, status=a.status)
        got.append(O)
    torch.cuda.synchronize()
    assert a.status.item() == 0
    for n, O in enumerate(got):
        assert (O == consts[n % len(consts)]).all(), n
    want = np.log(lens.double().cpu().numpy())[:, None]
    # a sum of ones is exact; log2 of up to 2^17 is off by two steps of 2^-19 at most, which ln 2
    # makes 2.6e-6, and the product by half a step of 2^-20
    assert np.abs(a.lse.double().cpu().numpy() - want).max() <= 2.0 ** -18
