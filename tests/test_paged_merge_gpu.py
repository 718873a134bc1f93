"""Decode attention over the paged 8-bit cache where a pair's tiles lie in many CTAs: every
listed block counts once, whatever its place, and every merge reads its own call's states."""
import numpy as np
import pytest
import torch

import paged_long as long
import paged_utils as ref
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


def cache(g, lens, H, extra=3):
    """Pages of random values, each block's of its own, and the tables that name them."""
    blocks = [-(-n // BLK) for n in lens]
    n_pages = sum(blocks) + extra
    pages = (torch.randn((n_pages, H, 2, BLK, D), generator=g, device=DEV) * 64).clamp(-448, 448).to(F8)
    scale = torch.full((n_pages, H, 2), 2.0 ** -7, device=DEV)
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return pages, scale, table


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("G", [1, 4, 8, 9, 16])
@pytest.mark.parametrize("H,lens", [(1, [20032]), (1, [40000]), (1, [131072]), (2, [131009]), (2, [131072, 77, 40001]),
                                    (1, [100000] * 5)])
def test_every_tile_of_a_long_list_counts_once(H, lens, G):
    """Queries of zero, so that all weights are 1, and values that are 1 in two of the 128 dims, which
    tell a block's number modulo 64 and 64 times that: O counts the tokens of each.  A tile that
    is lost or counted twice is 1 of at most 32 in its dims, and 5e-4 of exp(lse) at 131 072."""
    g = generator(G)
    pages, scale, table = cache(g, lens, H)
    scale.fill_(1.0)
    want = np.zeros((len(lens), D))
    for b, n in enumerate(lens):
        for j in range(-(-n // BLK)):
            rows = min(BLK, n - BLK * j)
            dims = [j % 64, 64 + j // 64 % 64]
            want[b, dims] += rows / n
    one_hot = torch.zeros((pages.shape[0], D), device=DEV)
    for b, n in enumerate(lens):
        j = torch.arange(-(-n // BLK), device=DEV)
        one_hot[table[b, j].long(), j % 64] = 1.0
        one_hot[table[b, j].long(), 64 + j // 64 % 64] = 1.0
    pages.view(torch.uint8)[:, :, 1] = one_hot.to(F8).view(torch.uint8)[:, None, None, :]
    Q = torch.zeros((len(lens), H * G, D), dtype=torch.bfloat16, device=DEV)
    a = Attn(len(lens), H * G, H)

    def call(idx=None, count=None):
        a.O.fill_(7.0)
        binding.sparse_paged_decode_attn_f8(Q, pages, scale, table, i32(lens), a.O, a.ws, blk_idx=idx, count=count, lse=a.lse,
                                            status=a.status)
        # sums of up to 2^17 ones, times 2^12, are exact; the quotient is rounded to bf16
        O, lse = a.O.double().cpu().numpy(), a.lse.double().cpu().numpy()
        assert (np.abs(O - want[:, None]) <= (2.0 ** -8 + 2.0 ** -20) * want[:, None]).all()
        assert np.abs(lse - np.log(lens)[:, None]).max() <= 2.0 ** -18   # as above
        assert a.status.item() == 0

    call()
    # the same blocks as lists, in another order for each pair
    k = table.shape[1]
    idx = torch.full((len(lens), H, k), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(lens):
        for h in range(H):
            idx[b, h, :-(-n // BLK)] = torch.randperm(-(-n // BLK), generator=g, device=DEV).to(torch.int32)
    call(idx, i32([[-(-n // BLK)] * H for n in lens]))


@pytest.mark.parametrize("G,H,n", [(16, 2, 131072), (8, 1, 40000), (4, 2, 20032), (9, 3, 70001)])
def test_every_block_of_a_long_list_is_found(G, H, n):
    """Keys of random signs, and each query along one block's key: its score is 64 above 0 in a list
    whose others stay below 30, so that O is that token's value.  Every block is asked for once."""
    g = generator(n)
    pages, scale, table = cache(g, [n], H)
    signs = torch.randint(0, 2, (pages.shape[0], H, BLK, D), generator=g, device=DEV) * 2 - 1
    pages[:, :, 0] = signs.float().to(F8)
    scale.fill_(1.0)
    blocks = -(-n // BLK)
    j = torch.arange(blocks, device=DEV)
    t = (7 * j + 3) % BLK
    t[-1] = min(int(t[-1]), n - 1 - BLK * (blocks - 1))
    key = signs[table[0].long(), :, t].float()                    # [blocks][H][128]
    value = pages.float()[table[0].long(), :, 1, t]
    a = Attn(1, H * G, H)
    lens, got = i32([n]), torch.empty((blocks, H, D), device=DEV)
    for j0 in range(0, blocks, G):
        take = torch.arange(j0, j0 + G, device=DEV) % blocks
        Q = key[take].transpose(0, 1).reshape(1, H * G, D).to(torch.bfloat16)
        binding.sparse_paged_decode_attn_f8(Q, pages, scale, table, lens, a.O, a.ws, scale=0.5, status=a.status)
        got[take] = a.O.view(H, G, D).transpose(0, 1).float()
    # the others weigh n * e^-34 < 2^-31 together; values of 4 bits are bf16's
    assert (got - value).abs().max() <= 2.0 ** -8 * 448 and ((got - value).abs() <= 2.0 ** -8 * value.abs() + 2.0 ** -21).all()
    assert a.status.item() == 0


@pytest.mark.parametrize("G", [1, 4, 8, 11, 16])
@pytest.mark.parametrize("H,lens", [(1, [20032]), (2, [40000]), (1, [131072]), (2, [131009, 33000, 131072])])
def test_attn_over_long_lists(H, lens, G):
    """Random values against the plain implementation, within a bound that a lost tile does not meet."""
    pages, scale, table = cache(generator(sum(lens) + G), lens, H)
    Q = torch.randn((len(lens), H * G, D), generator=generator(G), device=DEV).to(torch.bfloat16)
    a = Attn(len(lens), H * G, H)
    binding.sparse_paged_decode_attn_f8(Q, pages, scale, table, i32(lens), a.O, a.ws, lse=a.lse, status=a.status)
    torch.cuda.synchronize()
    values, scales, tables = ref.f8_values(pages), ref.f64(scale), table.cpu().numpy()
    O, lse, q = ref.f64(a.O), ref.f64(a.lse), ref.f64(Q)
    for b, n in enumerate(lens):
        for h in range(H):
            of = slice(h * G, (h + 1) * G)
            K, V = long.tokens(values, scales, tables[b], n, h)
            long.assert_close(O[b, of], lse[b, of], long.attend(q[b, of], K, V), f"request {b}, head {h}")
    assert a.status.item() == 0
