"""Chunk attention, rotary positions, forks and copies without a GPU: what the C calls and the binding
refuse before any launch, and the plain fork that the GPU is held to."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_long_pool_gb300 import binding, build, rope
from tests import chunk_utils as U

FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)   # never dereferenced
INVALID, UNSUPPORTED = binding.SPARSE_ERR_INVALID_ARG, binding.SPARSE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def calls(f, good, cases):
    for at, value, want in cases:
        args = list(good)
        args[at] = value
        assert f(*args) == want, (at, value, binding.load().sparse_last_error())


def test_chunk_attention_refuses(lib):
    # Q q_stride pages scale n_pages table max_blocks cu start n_tok B H_q H_kv scale O lse ws bytes status stream
    good = [FAKE, 1024, FAKE, FAKE, 10, FAKE, 8, FAKE, FAKE, 5, 2, 8, 2, 0.0, FAKE, FAKE, FAKE, 1 << 30, None, None]
    calls(lib.sparse_paged_chunk_attn_f8, good, [
        *((i, None, INVALID) for i in (0, 2, 3, 5, 7, 8, 14, 16)), *((i, ODD, INVALID) for i in (0, 2, 3, 5, 7, 8, 14, 15, 16)),
        (1, 1016, INVALID), (1, 1028, INVALID), (4, 0, INVALID), (6, 0, INVALID), (9, 0, INVALID), (10, 0, INVALID), (11, 7, INVALID),
        (12, 0, INVALID), (13, 3e38, INVALID), (13, float("nan"), INVALID),
        (10, 4097, UNSUPPORTED), (4, (1 << 25) + 1, UNSUPPORTED), (6, 1 << 25, UNSUPPORTED), (9, (1 << 30) + 1, UNSUPPORTED)])
    wide = list(good)
    wide[1], wide[11] = 34 * 128, 34
    assert lib.sparse_paged_chunk_attn_f8(*wide) == UNSUPPORTED   # 17 query heads a KV head
    assert lib.sparse_paged_chunk_attn_f8_workspace_size(0, 8, 2) == 0
    assert lib.sparse_paged_chunk_attn_f8_workspace_size(1, 34, 2) == 0


def test_rope_refuses(lib):
    # Q q_stride H_q K k_stride H_kv pos n_tok freq rot interleaved factor Q_out q_out_stride K_out k_out_stride stream
    good = [FAKE, 512, 4, FAKE, 128, 1, FAKE, 3, FAKE, 128, 0, 1.0, FAKE, 512, FAKE, 128, None]
    calls(lib.sparse_rope, good, [
        *((i, None, INVALID) for i in (0, 3, 6, 8, 12, 14)), *((i, ODD, INVALID) for i in (0, 3, 6, 8, 12, 14)),
        (1, 504, INVALID), (4, 120, INVALID), (13, 516, INVALID), (15, 0, INVALID), (2, 0, INVALID), (5, -1, INVALID), (7, 0, INVALID),
        (9, 0, INVALID), (9, 3, INVALID), (9, 130, INVALID), (11, float("inf"), INVALID), (11, float("nan"), INVALID),
        (7, (1 << 30) + 1, UNSUPPORTED)])


def test_fork_refuses(lib):
    # src fork_len B seq_len table max_blocks extra free n_pages n_free copy_src copy_dst ws bytes status stream
    good = [FAKE, None, 4, FAKE, FAKE, 9, FAKE, FAKE, 20, FAKE, FAKE, FAKE, FAKE, 1 << 20, None, None]
    calls(lib.sparse_page_fork, good, [
        *((i, None, INVALID) for i in (0, 3, 4, 6, 7, 9, 10, 11, 12)), *((i, ODD, INVALID) for i in (0, 1, 3, 4, 6, 7, 9, 10, 11, 12)),
        (2, 0, INVALID), (5, 0, INVALID), (8, 0, INVALID), (13, 100, INVALID),
        (2, 4097, UNSUPPORTED), (5, 1 << 25, UNSUPPORTED), (8, (1 << 25) + 1, UNSUPPORTED)])
    most = list(good)
    most[2], most[5] = 4096, (1 << 25) - 1
    assert lib.sparse_page_fork(*most) == UNSUPPORTED
    assert lib.sparse_page_fork_workspace_size(4097, 3) == 0 and lib.sparse_page_fork_workspace_size(4, 33) >= 4 * 4 * 2


def test_copy_refuses(lib):
    # pages scale n_pages H_kv copy_src copy_dst n_copy ktil B N_cap src seq_len status stream
    good = [FAKE, FAKE, 5, 2, FAKE, FAKE, 3, FAKE, 3, 4, FAKE, FAKE, None, None]
    calls(lib.sparse_paged_copy_f8, good, [
        *((i, None, INVALID) for i in (0, 1, 4, 5, 10, 11)), *((i, ODD, INVALID) for i in (0, 1, 4, 5, 7, 10, 11)),
        (2, 0, INVALID), (3, 0, INVALID), (6, 0, INVALID), (8, 0, INVALID), (9, 0, INVALID),
        (2, (1 << 25) + 1, UNSUPPORTED), (3, 65536, UNSUPPORTED), (8, 4097, UNSUPPORTED), (9, 1 << 25, UNSUPPORTED)])


def test_tensors_of_the_host_are_refused():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.sparse_page_fork(t, t, torch.zeros((4, 2), dtype=torch.int32), t, t, t, t, t, t)
    with pytest.raises(ValueError):
        binding.sparse_rope(torch.zeros((1, 1, 128), dtype=torch.bfloat16), None, t, t, t, None)
    with pytest.raises(TypeError):
        binding.sparse_paged_chunk_attn_f8(t, None, t, t, t, t, t, t)


def test_frequencies():
    f, factor = rope.frequencies(64)
    assert factor == 1.0 and f[0] == 1.0 and np.allclose(f, 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-15)
    g, _ = rope.frequencies(64, scaling="linear", scale=4.0)
    assert torch.equal(g, f / 4)
    g, _ = rope.frequencies(64, scaling="base", scale=4.0)
    assert g[0] == 1.0 and abs(g[-1] / f[-1] * 4 - 1) < 1e-12
    g, factor = rope.frequencies(64, scaling="parts", scale=8.0, original_len=2048)
    turns = 2048 * f / (2 * np.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.equal(g[turns < 1], f[turns < 1] / 8)
    assert ((g <= f) & (g >= f / 8)).all() and abs(factor - (0.1 * np.log(8) + 1)) < 1e-15
    for kw in ({"scaling": "other"}, {"scale": 0.0}, {"base": -1.0}, {"scaling": "parts", "slow_turns": 40.0}):
        with pytest.raises(ValueError):
            rope.frequencies(64, **kw)
    for r in (0, 3, 130):
        with pytest.raises(ValueError):
            rope.frequencies(r)


def test_plain_fork_keeps_the_books():
    rng = np.random.default_rng(1)
    B, N, n_pages = 12, 9, 150
    lens = [int(x) for x in rng.integers(0, 64 * N + 1, B)]
    perm = rng.permutation(n_pages)
    table = np.full((B, N), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        table[b, : U.nblk(n)] = perm[at : at + U.nblk(n)]
        at += U.nblk(n)
    free = np.full(n_pages, -1, np.int32)
    free[: n_pages - at] = perm[at:]
    extra, n_free = np.zeros(n_pages, np.int32), n_pages - at
    for _ in range(20):
        src = np.arange(B)
        keep = rng.choice(B, 6, replace=False)
        for b in set(range(B)) - set(keep.tolist()):
            src[b] = rng.choice([-1, *keep])
        r = U.fork(src, lens, table, extra, free, n_free)
        table, extra, free, n_free, lens = r["table"], r["extra"], r["free"], r["n_free"], r["len"].tolist()
        held = np.zeros(n_pages, int)
        for b, n in enumerate(lens):
            for j in range(U.nblk(n)):
                held[table[b, j]] += 1
        listed = free[:n_free]
        assert len(set(listed.tolist())) == n_free and (held[listed] == 0).all() and (held > 0).sum() + n_free == n_pages
        assert np.array_equal(np.maximum(held - 1, 0), extra)
