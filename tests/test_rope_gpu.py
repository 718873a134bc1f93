"""Rotary positions against 64 bits."""
import pytest
import torch

from block_sparse_long_pool_gb300 import binding, rope
from tests import chunk_utils as U

pytestmark = pytest.mark.gpu


def rows(n, H, seed, strided):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, (H + 3 if strided else H) * 128), generator=g, device="cuda").to(torch.bfloat16)
    return x[:, : H * 128].view(n, H, 128) if not strided else x[:, 256 : 256 + H * 128].view(n, H, 128)


def check(x, got, pos, f, inter, factor, fill=0.0):
    want, size = U.rope(x, pos, f, inter, factor)
    want = torch.where((pos >= 0)[:, None, None], want, fill)
    # bf16's half step, fp32 products and sum (3 roundings of the parts), angles to 2^-23 turns in fp32 and 2^-21 by sincospi
    tol = want.abs() * 2.0 ** -8 + size * (2.0 ** -18) * (1 + 2.0 ** -8)
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (err / tol.clamp(min=1e-30)).max().item()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [2, 6, 16, 20, 64, 80, 96, 126, 128])
@pytest.mark.parametrize("n,H_q,H_kv", [(1, 1, 1), (7, 8, 2), (33, 5, 5), (1500, 20, 4)])
def test_layouts(inter, rot, n, H_q, H_kv):
    Q, K = rows(n, H_q, 1, True), rows(n, H_kv, 2, n % 2 == 0)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(0, 200000, (n,), generator=g, device="cuda").to(torch.int32)
    if n > 2:
        pos[1] = -1
        pos[n - 1] = -5
        pos[0] = 0
    f, factor = rope.frequencies(rot, base=10000.0)
    f = f.cuda()
    Qo, Ko = torch.full_like(Q, 3.0, memory_format=torch.contiguous_format), torch.full((n, H_kv, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    binding.sparse_rope(Q, K, pos, f, Qo, Ko, interleaved=inter, factor=1.3)
    check(Q, Qo, pos, f, inter, 1.3, fill=3.0)
    check(K, Ko, pos, f, inter, 1.3, fill=3.0)
    # in place, queries alone
    X = Q.clone(memory_format=torch.contiguous_format)
    binding.sparse_rope(X, None, pos, f, X, None, interleaved=inter, factor=1.3)
    live = pos >= 0
    assert torch.equal(X[live], Qo[live]) and torch.equal(X[~live], Q[~live])


@pytest.mark.parametrize("n", [9, 5000])
def test_far_positions(n):
    Q = rows(n, 2, 5, False)
    g = torch.Generator(device="cuda").manual_seed(6)
    pos = torch.randint(2 ** 31 - 10 ** 6, 2 ** 31, (n,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    f = torch.cat([rope.frequencies(126)[0], torch.tensor([3.5])]).cuda()
    out = torch.empty_like(Q)
    binding.sparse_rope(Q, None, pos, f, out, None)
    # the reference's own angles: the product in 64 bits is off by 2^-22 radian there
    want, size = U.rope(Q, pos, f, False, 1.0)
    assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2.0 ** -17).all()


def test_negative_and_large_frequencies():
    Q = rows(40, 2, 7, False)
    pos = torch.arange(40, dtype=torch.int32, device="cuda") * 997
    f = torch.tensor([-1.0, 0.0, 7.25, -2.5, 100.0, 1e-9, 6.283185307179586, 0.5], dtype=torch.float64, device="cuda")
    out = torch.empty_like(Q)
    binding.sparse_rope(Q, None, pos, f, out, None)
    check(Q, out, pos, f, False, 1.0)


def test_frequencies():
    f, s = rope.frequencies(128)
    assert f.dtype == torch.float64 and f[0] == 1 and s == 1.0
    assert torch.allclose(f, 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128))


def test_captured_and_on_a_stream():
    Q, K = rows(200, 8, 8, True), rows(200, 2, 9, True)
    pos = torch.arange(200, dtype=torch.int32, device="cuda")
    f = rope.frequencies(128)[0].cuda()
    Qo, Ko = torch.empty((200, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((200, 2, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    binding.sparse_rope(Q, K, pos, f, Qo, Ko, stream=s)
    s.synchronize()
    check(Q, Qo, pos, f, False, 1.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.sparse_rope(Q, K, pos, f, Qo, Ko)
    pos += 1000
    g.replay()
    torch.cuda.synchronize()
    check(Q, Qo, pos, f, False, 1.0)
    check(K, Ko, pos, f, False, 1.0)


def test_refusals():
    Q, K = rows(4, 2, 1, False), rows(4, 1, 1, False)
    pos, f = torch.zeros(4, dtype=torch.int32, device="cuda"), rope.frequencies(128)[0].cuda()
    ok = [Q, K, pos, f, torch.empty_like(Q), torch.empty_like(K)]

    def refused(i, t, err, **kw):
        a = list(ok)
        if i is not None:
            a[i] = t
        with pytest.raises(err):
            binding.sparse_rope(*a, **kw)

    refused(0, Q.float(), TypeError)
    refused(1, K[:3], ValueError)
    refused(1, None, ValueError)
    refused(2, pos.long(), TypeError)
    refused(3, f.float(), TypeError)
    refused(3, torch.zeros(65, dtype=torch.float64, device="cuda"), binding.SparsePoolError)
    refused(3, torch.zeros(0, dtype=torch.float64, device="cuda"), binding.SparsePoolError)
    refused(4, Q[:, :1], ValueError)
    refused(5, K.transpose(0, 2), ValueError)
    refused(None, None, binding.SparsePoolError, factor=float("inf"))
