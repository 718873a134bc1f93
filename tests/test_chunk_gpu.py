"""Attention of a step's new rows over the paged cache against 64 bits."""
import pytest
import torch

from block_sparse_long_pool_gb300 import binding
from tests.chunk_utils import BLK, D, Chunk

pytestmark = pytest.mark.gpu


def ws(c):
    return binding.paged_chunk_workspace(c.B, c.H_q, c.H_kv)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 11, 16])
@pytest.mark.parametrize("start,new", [
    ([0], [1]), ([0], [64]), ([0], [129]), ([63], [2]), ([64], [1]), ([127], [130]), ([1000], [37]),
    ([0, 200, 0, 77], [0, 5, 300, 0]),
    ([5, -1, 640, -1], [40, 9, 1, 0]),
])
def test_lengths_and_heads(G, start, new):
    c = Chunk(start, new, 2, G, seed=G, pad=3)
    c.call(ws(c))
    c.check()


@pytest.mark.parametrize("start,new,H,G", [
    ([40000], [5], 1, 4), ([33000], [300], 2, 4), ([9000, 20000, 1], [1, 1, 1], 2, 8), ([0], [3000], 2, 1), ([6000] * 20, [1] * 20, 1, 16),
    ([3, 0, 12345, 700] * 6, [1, 260, 1, 33] * 6, 2, 5),
])
def test_long_and_split(start, new, H, G):
    c = Chunk(start, new, H, G, seed=3, strided=True)
    c.call(ws(c))
    c.check()


def test_rows_outside_are_left_as_they_were():
    c = Chunk([100, 4000], [70, 33], 2, 4, first=5, pad=40)
    c.call(ws(c))
    c.check()   # rows before cu_new[0] and behind the last request: 7, as filled
    assert (c.O[:5] == 7).all() and (c.O[-40:] == 7).all() and (c.lse[-40:] == 7).all()


@pytest.mark.parametrize("scale", [0.02, -0.11, 3.0])
def test_scales(scale):
    c = Chunk([500], [90], 2, 4, seed=5)
    c.call(ws(c), scale=scale)
    c.check(scale)


@pytest.mark.parametrize("exps,q_mag", [((-60, -20), 1e-3), ((-110, -90), 1.0), ((-30, 40), 1e-12), ((-7, -5), 2.0 ** -90)])
def test_page_scales_far_apart(exps, q_mag):
    c = Chunk([3000, 100], [50, 20], 2, 4, seed=6, exps=exps, q_mag=q_mag)
    if exps[1] - exps[0] > 5:   # keys alike, so that every page counts; values far apart
        c.scale[..., 0] = 2.0 ** -6
    c.call(ws(c))
    c.check()


def test_values_outweigh_scores():
    # scores fall by 2^120 from page to page while value scales grow by as much
    c = Chunk([640], [20], 1, 4, seed=7)
    c.pages.copy_((c.pages.float().nan_to_num() / 8).to(torch.float8_e4m3fn))
    c.Q.zero_()
    c.Q[..., 0] = 1.0
    for j in range(11):
        p = int(c.table[0, j])
        c.pages[p, :, 0, :, 0] = 8.0
        c.pages[p, :, 0, :, 1:] = 0.0
        c.scale[p, :, 0] = 16.0 - j
        c.scale[p, :, 1] = 2.0 ** (-100 + 20 * j)
    c.call(ws(c), scale=1.0)
    c.check(1.0)


def test_zero_scales():
    c = Chunk([300], [30], 1, 2, seed=8)
    c.scale[int(c.table[0, 0])] = 0.0
    c.scale[int(c.table[0, 3]), :, 1] = 0.0
    c.call(ws(c))
    c.check()
    c.scale.zero_()
    c.call(ws(c))
    c.check()


def test_nan_values_reach_the_rows_that_see_them():
    c = Chunk([100, 0, 9000], [200, 128, 3], 2, 4, seed=9)
    nan = float("nan")
    for b, tok, h, d in [(0, 150, 0, 5), (0, 299, 1, 127), (0, 20, 1, 64), (1, 64, 0, 0), (1, 127, 1, 33), (2, 8999, 0, 9)]:
        c.pages[int(c.table[b, tok // BLK]), h, 1, tok % BLK, d] = nan
    c.pages[int(c.table[1, 1]), 0, 0, 10, 3] = nan   # a key: every dim of the rows that see it
    c.call(ws(c))
    c.check()
    assert c.O.isnan().any()


def test_nan_is_of_its_item():
    # many short requests a CTA, one of them with NaN
    n = 400
    c = Chunk([i % 130 for i in range(n)], [1 + i % 3 for i in range(n)], 1, 4, seed=10)
    for b in (7, 150):
        c.pages[int(c.table[b, 0]), 0, 1, 0, b % D] = float("nan")
    c.call(ws(c))
    c.check()


def test_queries_with_nan_and_infinity():
    c = Chunk([70], [60], 1, 4, seed=11)
    c.Q[3, 1, 5] = float("nan")
    c.call(ws(c))
    torch.cuda.synchronize()
    assert c.O[3, 1].isnan().all() and c.lse[3, 1].isnan()
    keep = c.Q[3, 1].clone()
    c.Q[3, 1] = c.Q[3, 0]
    O, lse = c.O.clone(), c.lse.clone()
    c.call(ws(c))
    c.check()
    c.Q[3, 1] = keep
    ok = torch.ones_like(c.lse, dtype=torch.bool)
    ok[3, 1] = False
    assert torch.equal(O[ok], c.O[ok]) and torch.equal(lse[ok], c.lse[ok])


def test_bad_pages_and_lengths_are_reported():
    c = Chunk([300, 50], [40, 6], 1, 4, seed=12)
    c.table[0, 2] = c.n_pages
    c.table[0, 4] = -3
    c.call(ws(c))
    c.check(status=binding.SPARSE_ERR_BAD_INDEX)
    c = Chunk([300], [100], 1, 4, seed=13, extra_blocks=0)
    c.start.fill_(380)   # the table holds 448 tokens: the last rows are past it
    c.call(ws(c))
    c.check(status=binding.SPARSE_ERR_BAD_INDEX)
    c = Chunk([10, 20], [5, 6], 1, 4, seed=14)
    c.cu.copy_(torch.tensor([0, 5, 400], device="cuda"))
    c.call(ws(c))
    torch.cuda.synchronize()
    assert c.status.item() == binding.SPARSE_ERR_BAD_INDEX
    c.cu.copy_(torch.tensor([0, 5, 11], device="cuda"))
    c.status.zero_()
    c.check()


def test_every_page_bad():
    c = Chunk([300], [40], 1, 4, seed=15)
    c.table.fill_(-1)
    c.call(ws(c))
    c.check(status=binding.SPARSE_ERR_BAD_INDEX)
    assert (c.O == 0).all() and c.lse.isinf().all()


def test_no_rows():
    c = Chunk([0, 0], [0, 0], 1, 4, pad=10)
    c.call(ws(c))
    c.check()
    assert (c.O == 7).all()


def test_many_requests():
    n = 4096
    c = Chunk([(i * 37) % 300 if i % 5 else -1 for i in range(n)], [1 if i % 3 else 0 for i in range(n)], 1, 2, seed=16, pad=7)
    c.call(ws(c))
    c.check()


def test_shared_workspace_streams_and_the_same_bits():
    a, b = Chunk([20000, 3], [9, 500], 2, 4, seed=17), Chunk([100] * 30, [20] * 30, 1, 5, seed=18)
    w = max((ws(a), ws(b)), key=lambda t: t.numel())
    w.fill_(255)
    for _ in range(2):
        a.call(w)
        b.call(w)
    a.check()
    b.check()
    O, lse = a.O.clone(), a.lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        a.call(w, stream=s)
        s.synchronize()
        assert torch.equal(O, a.O) and torch.equal(lse, a.lse)
    # two calls at once, each with a workspace of its own
    w2 = ws(b)
    a.O.fill_(0)
    b.O.fill_(0)
    torch.cuda.synchronize()
    for _ in range(5):
        a.call(w, stream=s)
        b.call(w2)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_captured_as_lengths_change():
    c = Chunk([500, 100], [30, 40], 2, 4, seed=19)
    w = ws(c)
    c.call(w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(w)
    for start in ([500, 100], [200, 0], [-1, 90]):
        c.start.copy_(torch.tensor(start, dtype=torch.int32))
        c.O.fill_(7)
        c.lse.fill_(7)
        g.replay()
        c.check()


def test_single_tokens_as_the_decode_call():
    B, H, G = 5, 2, 4
    c = Chunk([63, 64, 900, 0, 20000], [1] * B, H, G, seed=20)
    c.call(ws(c))
    O = torch.empty_like(c.O)
    binding.sparse_paged_decode_attn_f8(c.Q.contiguous(), c.pages, c.scale, c.table, c.start + 1, O, binding.paged_workspace(B, H * G, H))
    c.check()
    _, _, tol, _ = c.expected()
    assert ((O.double() - c.O.double()).abs() <= 2 * tol).all()


def test_cache_past_4gb():
    c = Chunk([200], [30], 4, 4, seed=21)
    n = (1 << 32) // (4 * 2 * BLK * D) + 100
    pages = torch.zeros((n, 4, 2, BLK, D), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.zeros((n, 4, 2), device="cuda")
    pages[n - c.n_pages:] = c.pages
    scale[n - c.n_pages:] = c.scale
    c.table = torch.where(c.table >= 0, c.table + (n - c.n_pages), c.table)
    c.pages, c.scale, c.n_pages = pages, scale, n
    c.call(ws(c))
    c.check()


def test_refusals():
    c = Chunk([10], [4], 2, 4)
    w = ws(c)
    call = binding.sparse_paged_chunk_attn_f8
    args = [c.Q, c.pages, c.scale, c.table, c.cu, c.start, c.O, w]

    def refused(i, t, err, **kw):
        a = list(args)
        if i is not None:
            a[i] = t
        with pytest.raises(err):
            call(*a, **kw)

    refused(0, c.Q.float(), TypeError)
    refused(0, c.Q[:, :7], ValueError)
    refused(0, c.Q.transpose(1, 2).contiguous().transpose(1, 2), ValueError)
    refused(1, c.pages.view(torch.uint8), TypeError)
    refused(2, c.scale[:-1], ValueError)
    refused(3, c.table.long(), TypeError)
    refused(4, c.cu[:-1], ValueError)
    refused(5, c.start.cpu(), ValueError)
    refused(6, c.O[:-1], ValueError)
    refused(7, w[:1000], binding.SparsePoolError)
    refused(None, None, binding.SparsePoolError, scale=3e38)
    refused(None, None, ValueError, lse=c.lse[:, :3])
    refused(None, None, TypeError, status=torch.zeros(1, device="cuda"))
    q = torch.zeros((4, 17 * 2, D), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.SparsePoolError):
        call(q, *args[1:6], torch.empty_like(q), w)
