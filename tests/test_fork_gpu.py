"""Forked and ended requests that share pages, and what a fork copies."""
import numpy as np
import pytest
import torch

from block_sparse_long_pool_gb300 import binding
from tests import chunk_utils as U

pytestmark = pytest.mark.gpu


class Pool:
    def __init__(self, lens, max_blocks, n_pages, seed=0):
        rng = np.random.default_rng(seed)
        perm = rng.permutation(n_pages).astype(np.int32)
        table = np.full((len(lens), max_blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(lens):
            table[b, : U.nblk(n)] = perm[at : at + U.nblk(n)]
            at += U.nblk(n)
        free = np.full(n_pages, -1, np.int32)
        free[: n_pages - at] = perm[at:]
        t = lambda v: torch.tensor(np.asarray(v, np.int32), device="cuda")
        B = len(lens)
        self.B = B
        self.table, self.lens, self.extra, self.free, self.n_free = t(table), t(lens), t(np.zeros(n_pages)), t(free), t([n_pages - at])
        self.copy_src, self.copy_dst, self.status = t(np.zeros(B)), t(np.zeros(B)), t([0])
        self.ws = binding.page_fork_workspace(B, max_blocks)

    def call(self, src, fork_len=None, **kw):
        t = lambda v: None if v is None else torch.tensor(np.asarray(v, np.int32), device="cuda")
        binding.sparse_page_fork(t(src), self.lens, self.table, self.extra, self.free, self.n_free, self.copy_src, self.copy_dst, self.ws,
                                 fork_len=t(fork_len), status=self.status, **kw)

    def step(self, src, fork_len=None):
        n = lambda v: v.cpu().numpy()
        want = U.fork(src, n(self.lens), n(self.table), n(self.extra), n(self.free), int(self.n_free), fork_len)
        self.status.zero_()
        self.call(src, fork_len)
        for k, got in dict(table=self.table, extra=self.extra, free=self.free, n_free=self.n_free, len=self.lens, copy_src=self.copy_src,
                           copy_dst=self.copy_dst).items():
            assert np.array_equal(n(got).reshape(-1), np.asarray(want[k]).reshape(-1)), k
        assert self.status.item() == (binding.SPARSE_ERR_NO_PAGES if want["refused"] else 0)
        return want


def sources(rng, B, p_end=0.2, p_fork=0.4):
    stay = rng.random(B) > p_end + p_fork
    stay[rng.integers(B)] = True
    keep = np.flatnonzero(stay)
    src = np.arange(B)
    for b in np.flatnonzero(~stay):
        src[b] = -1 if rng.random() < p_end / (p_end + p_fork) else rng.choice(keep)
    return src


@pytest.mark.parametrize("B,T,max_blocks", [(1, 100, 4), (2, 64, 1), (3, 1, 1), (5, 700, 11), (33, 3000, 60), (100, 9000, 400), (257, 5000, 200), (4096, 90, 2)])
def test_steps(B, T, max_blocks):
    rng = np.random.default_rng(B)
    lens = [int(rng.integers(0, min(T, 64 * max_blocks) + 1)) for _ in range(B)]
    pool = Pool(lens, max_blocks, sum(U.nblk(n) for n in lens) + B + 3, seed=B)
    for i in range(6):
        src = sources(rng, B)
        fl = None if i % 2 else rng.integers(-1, T + 100, B)
        pool.step(src, fl)
    pool.step(np.full(B, -1))   # everything ends: every page is free
    assert int(pool.n_free) == pool.free.numel() and (pool.extra == 0).all()
    assert sorted(pool.free.tolist()) == list(range(pool.free.numel()))


def test_too_few_pages():
    pool = Pool([100, 0, 0, 0, 64, 0], 4, 5, seed=1)
    want = pool.step([0, 0, 0, 0, 4, 4])   # two pages left: the third sample of 100 tokens gets none
    assert want["refused"] == 1 and pool.lens.tolist() == [100, 100, 100, 0, 64, 64]
    pool.step([0, -1, 2, 0, 4, 5])


def test_shared_page_outlives_its_first_owner():
    pool = Pool([128, 0, 0], 2, 6)
    pool.step([0, 0, 0])
    a = pool.table[0].tolist()
    pool.step([-1, 1, 2])
    assert pool.table[1].tolist() == a and pool.extra[a].tolist() == [1, 1]
    pool.step([-1, 1, 1])
    pool.step([0, 1, -1])
    assert pool.extra[a].tolist() == [0, 0]
    pool.step([0, -1, 2])
    assert int(pool.n_free) == 6


def test_unsound_inputs_are_reported():
    for src, want in [([1, 0, 2], [130, 70, 5]), ([0, 7, 2], [130, 70, 5]), ([0, 2, 0], [130, 70, 130])]:
        pool = Pool([130, 70, 5], 3, 12)
        pool.call(src)   # a source that does not stay, or is outside: that request stays as it is
        torch.cuda.synchronize()
        assert pool.status.item() == binding.SPARSE_ERR_BAD_INDEX and pool.lens.tolist() == want
    pool = Pool([130, 70, 5], 3, 12)
    pool.lens[1] = 1000
    before = int(pool.n_free)
    pool.call([0, 1, 1])   # a copy of a request whose length is unsound ends
    torch.cuda.synchronize()
    assert pool.status.item() == binding.SPARSE_ERR_BAD_INDEX and pool.lens.tolist() == [130, 1000, 0] and int(pool.n_free) == before + 1
    pool = Pool([130, 70, 5], 3, 12)
    pool.lens[1] = -4
    before = int(pool.n_free)
    pool.call([0, -1, 1])   # it gives up no pages; a copy of it stays as it was, since it does not
    torch.cuda.synchronize()
    assert pool.status.item() == binding.SPARSE_ERR_BAD_INDEX and pool.lens.tolist() == [130, 0, 5] and int(pool.n_free) == before
    pool = Pool([130, 70, 5], 3, 12)
    pool.table[1, 0] = 99
    before = int(pool.n_free)
    pool.call([0, -1, 2])
    torch.cuda.synchronize()
    assert pool.status.item() == binding.SPARSE_ERR_BAD_INDEX and int(pool.n_free) == before + 1
    pool = Pool([130, 70, 5], 3, 12)
    pool.n_free.fill_(50)
    pool.call([0, -1, 2])
    torch.cuda.synchronize()
    assert pool.status.item() == binding.SPARSE_ERR_BAD_INDEX and int(pool.n_free) == 12


def test_captured():
    pool = Pool([100, 0, 0, 0], 3, 12)
    src = torch.tensor([0, 0, 0, 0], dtype=torch.int32, device="cuda")
    end = torch.tensor([0, -1, -1, -1], dtype=torch.int32, device="cuda")
    args = (pool.lens, pool.table, pool.extra, pool.free, pool.n_free, pool.copy_src, pool.copy_dst, pool.ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.sparse_page_fork(src, *args, status=pool.status)
        binding.sparse_page_fork(end, *args, status=pool.status)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert pool.lens.tolist() == [100, 0, 0, 0] and pool.status.item() == 0 and (pool.extra == 0).all()
    assert sorted(pool.free[: int(pool.n_free)].tolist() + pool.table[0, :2].tolist()) == list(range(12))


@pytest.mark.parametrize("B,H,N,n_pages", [(1, 1, 1, 3), (4, 2, 5, 9), (40, 8, 70, 90), (300, 1, 33, 700)])
def test_copy(B, H, N, n_pages):
    rng = np.random.default_rng(B)
    g = torch.Generator(device="cuda").manual_seed(B)
    pages = torch.randint(0, 256, (n_pages, H, 2, 64, 128), generator=g, device="cuda").to(torch.uint8)
    scale = torch.rand((n_pages, H, 2), generator=g, device="cuda")
    ktil = torch.randn((B, H, N, 128), generator=g, device="cuda")
    src = sources(rng, B)
    lens = rng.integers(0, 64 * N + 1, B)
    lens[rng.integers(B)] = 0
    perm = rng.permutation(n_pages)
    a, z = np.full(B, -1), np.full(B, -1)
    for b in range(B):
        if src[b] not in (b, -1) and rng.random() < 0.8:
            a[b], z[b] = perm[0], perm[1 + b]
    want_p, want_s, want_k = pages.clone(), scale.clone(), ktil.clone()
    for b in range(B):
        if z[b] >= 0:
            want_p[z[b]], want_s[z[b]] = pages[a[b]], scale[a[b]]
        if 0 <= src[b] != b:
            n = U.nblk(int(lens[b]))
            want_k[b, :, :n] = ktil[src[b], :, :n]
    t = lambda v: torch.tensor(np.asarray(v, np.int32), device="cuda")
    status = t([0])
    got_p, got_s, got_k = pages.clone(), scale.clone(), ktil.clone()
    binding.sparse_paged_copy_f8(got_p.view(torch.float8_e4m3fn), got_s, t(a), t(z), ktil=got_k, src=t(src), seq_len=t(lens), status=status)
    assert torch.equal(got_p, want_p) and torch.equal(got_s, want_s) and torch.equal(got_k, want_k) and status.item() == 0
    got_p, got_s = pages.clone(), scale.clone()
    binding.sparse_paged_copy_f8(got_p.view(torch.float8_e4m3fn), got_s, t(a), t(z))
    assert torch.equal(got_p, want_p) and torch.equal(got_s, want_s)


def test_copy_reports_what_is_outside():
    pages = torch.zeros((3, 1, 2, 64, 128), device="cuda").to(torch.float8_e4m3fn)
    scale, ktil = torch.rand((3, 1, 2), device="cuda"), torch.randn((3, 1, 2, 128), device="cuda")
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    before = scale.clone(), ktil.clone()
    for a, z, src, lens in [([0], [3], [0, 1, 2], [1, 1, 1]), ([-1], [0], [0, 1, 2], [1, 1, 1]), ([0], [-1], [0, 1, 2], [1, 1, 1]),
                            ([-1], [-1], [0, 2, 0], [1, 1, 0]), ([-1], [-1], [0, 0, 5], [1, 0, 1]), ([-1], [-1], [0, 0, 2], [1, 129, 1])]:
        status = t([0])
        binding.sparse_paged_copy_f8(pages, scale, t(a), t(z), ktil=ktil, src=t(src), seq_len=t(lens), status=status)
        assert status.item() == binding.SPARSE_ERR_BAD_INDEX
        assert torch.equal(scale, before[0]) and torch.equal(ktil, before[1])


def test_refusals():
    pool = Pool([100, 0], 3, 12)
    src = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    ok = [src, pool.lens, pool.table, pool.extra, pool.free, pool.n_free, pool.copy_src, pool.copy_dst, pool.ws]
    for i, t, err in [(0, src.long(), TypeError), (1, pool.lens[:1], ValueError), (3, pool.extra[:5], ValueError), (5, pool.free, ValueError),
                      (8, pool.ws[:16], binding.SparsePoolError), (2, pool.table.t(), ValueError)]:
        a = list(ok)
        a[i] = t
        with pytest.raises(err):
            binding.sparse_page_fork(*a)
    pages = torch.zeros((3, 1, 2, 64, 128), device="cuda").to(torch.float8_e4m3fn)
    scale = torch.zeros((3, 1, 2), device="cuda")
    with pytest.raises(ValueError):
        binding.sparse_paged_copy_f8(pages, scale, src, src, ktil=torch.zeros((2, 1, 4, 128), device="cuda"))
    with pytest.raises(ValueError):
        binding.sparse_paged_copy_f8(pages, scale, src, src[:1])
