"""The paged 8-bit cache's calls without a GPU: what they refuse, and the plain
implementations that the GPU tests compare with, held to small cases worked by hand."""
import ctypes

import numpy as np
import pytest
import torch

import paged_utils as ref
from block_sparse_long_pool_gb300 import binding, build

FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10004)
INVALID, UNSUPPORTED = binding.SPARSE_ERR_INVALID_ARG, binding.SPARSE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


PLAN = dict(seq_len=FAKE, n_new=FAKE, B=4, table=FAKE, max_blocks=8, free=FAKE, n_pages=32, n_free=FAKE, cu=FAKE, start=FAKE,
            len_out=FAKE, n_free_out=FAKE, slot=FAKE, req=FAKE, pos=FAKE, n_tok=16, status=None, stream=None)
APPEND = dict(pages=FAKE, scale=FAKE, n_pages=32, H=2, k=FAKE, v=FAKE, ks=256, vs=256, slot=FAKE, n_tok=16, ktil=FAKE, B=4,
              N_cap=8, req=FAKE, pos=FAKE, status=None, stream=None)
ATTN = dict(Q=FAKE, pages=FAKE, scale=FAKE, n_pages=32, table=FAKE, max_blocks=8, idx=FAKE, count=FAKE, k_tot=6, len=FAKE, B=4,
            H_q=8, H_kv=2, sm=0.0, O=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 30, status=None, stream=None)


@pytest.mark.parametrize("name,good,change,code", [
    *[("sparse_page_plan", PLAN, {x: None}, INVALID) for x, y in PLAN.items() if y is FAKE],
    *[("sparse_page_plan", PLAN, {x: ODD}, INVALID) for x in ("seq_len", "table", "slot")],
    *[("sparse_page_plan", PLAN, {x: 0}, INVALID) for x in ("B", "max_blocks", "n_pages", "n_tok")],
    ("sparse_page_plan", PLAN, {"B": 4097}, UNSUPPORTED),
    ("sparse_page_plan", PLAN, {"n_pages": (1 << 25) + 1}, UNSUPPORTED),
    ("sparse_page_plan", PLAN, {"max_blocks": (1 << 25) + 1}, UNSUPPORTED),
    ("sparse_page_plan", PLAN, {"n_tok": (1 << 30) + 1}, UNSUPPORTED),
    ("sparse_paged_append_f8", APPEND, {"n_tok": (1 << 30) + 1}, UNSUPPORTED),
    *[("sparse_paged_append_f8", APPEND, {x: None}, INVALID) for x in ("pages", "scale", "k", "v", "slot", "req", "pos")],
    *[("sparse_paged_append_f8", APPEND, {x: ODD}, INVALID) for x in ("pages", "scale", "k", "v", "slot", "ktil", "req", "pos")],
    *[("sparse_paged_append_f8", APPEND, {x: 0}, INVALID) for x in ("n_pages", "H", "n_tok", "B", "N_cap")],
    *[("sparse_paged_append_f8", APPEND, {x: y}, INVALID) for x in ("ks", "vs") for y in (255, 248, 260, -256, 0)],
    ("sparse_paged_append_f8", APPEND, {"n_pages": (1 << 25) + 1}, UNSUPPORTED),
    ("sparse_paged_append_f8", APPEND, {"H": 65536, "ks": 65536 * 128, "vs": 65536 * 128}, UNSUPPORTED),
    *[("sparse_paged_decode_attn_f8", ATTN, {x: None}, INVALID)
      for x in ("Q", "pages", "scale", "table", "count", "len", "O", "ws")],
    *[("sparse_paged_decode_attn_f8", ATTN, {x: ODD}, INVALID)
      for x in ("Q", "pages", "scale", "table", "idx", "count", "len", "O", "lse", "ws")],
    *[("sparse_paged_decode_attn_f8", ATTN, {x: 0}, INVALID) for x in ("B", "H_q", "H_kv", "n_pages", "max_blocks", "k_tot")],
    ("sparse_paged_decode_attn_f8", ATTN, {"H_q": 7}, INVALID),
    ("sparse_paged_decode_attn_f8", ATTN, {"H_q": 34}, UNSUPPORTED),
    ("sparse_paged_decode_attn_f8", ATTN, {"B": 32768}, UNSUPPORTED),
    ("sparse_paged_decode_attn_f8", ATTN, {"sm": float("nan")}, INVALID),
    ("sparse_paged_decode_attn_f8", ATTN, {"sm": float("inf")}, INVALID),
    ("sparse_paged_decode_attn_f8", ATTN, {"n_pages": (1 << 25) + 1}, UNSUPPORTED),
    # 128 pairs of 2^24 places each, 8 of them a pair's own: 2^31 in all
    ("sparse_paged_decode_attn_f8", ATTN, {"B": 64, "k_tot": (1 << 24) - 8}, UNSUPPORTED),
    ("sparse_paged_decode_attn_f8", ATTN, {"B": 64, "idx": None, "count": None, "max_blocks": (1 << 24) - 8}, UNSUPPORTED),
    ("sparse_paged_decode_attn_f8", ATTN, {"max_blocks": 1 << 25}, UNSUPPORTED),
    ("sparse_paged_decode_attn_f8", ATTN, {"k_tot": (1 << 25) + 1}, UNSUPPORTED),
    ("sparse_paged_decode_attn_f8", ATTN, {"n_pages": 1 << 25, "B": 1, "H_q": 32, "H_kv": 32}, UNSUPPORTED)])
def test_refusals(lib, name, good, change, code):
    args = {**good, **change}
    assert getattr(lib, name)(*args.values()) == code
    assert lib.sparse_last_error().decode().startswith(name)


def test_workspace_size_of_invalid_sizes(lib):
    f = lib.sparse_paged_decode_attn_f8_workspace_size
    for bad in ((0, 8, 2), (1, 7, 2), (1, 34, 2), (32768, 4, 2), (1, 8, 0)):
        assert f(*bad) == 0


def test_binding_refuses_other_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sparse_page_plan(i, i, i.view(4, 1), i, i[:1], i, i, i, i[:1], i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sparse_paged_append_f8(torch.zeros((1, 1, 2, 64, 128)).to(torch.float8_e4m3fn), None, None, None, i)
    with pytest.raises(TypeError):
        binding.sparse_paged_decode_attn_f8(None, None, None, None, None, None, None)


def test_plain_plan_by_hand():
    table = np.array([[3, -1], [5, 6], [-1, -1]], np.int32)
    got = ref.plan([64, 70, 0], [2, -1, 3], table, np.array([1, 2, 0, 0, 0, 0, 0], np.int32), 2, 6)
    # request 1 returns 5 and 6; request 0 takes 6 for its second block, request 2 takes 5
    assert got["table"].tolist() == [[3, 6], [5, 6], [5, -1]] and got["n_free"] == 2
    assert got["free"].tolist() == [1, 2, 5, 6, 0, 0, 0]
    assert got["slot"].tolist() == [6 * 64, 6 * 64 + 1, 5 * 64, 5 * 64 + 1, 5 * 64 + 2, -1]
    assert got["len"].tolist() == [66, 0, 3] and got["start"].tolist() == [64, 0, 0]


def test_plain_rounding_is_e4m3():
    grid = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    grid = np.unique(grid[np.isfinite(grid)])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 2000), rng.standard_normal(2000) * 2.0 ** -6, (grid[1:] + grid[:-1]) / 2, grid])
    want = torch.as_tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    x32 = torch.as_tensor(x, dtype=torch.float32).double().numpy()
    assert np.array_equal(ref.e4m3_round(x32), want)
    assert ref.pow2_scale(448.0) == 1 and ref.pow2_scale(448.5) == 2 and ref.pow2_scale(224.0) == 0.5
    assert ref.pow2_scale(0.0) == 2.0 ** -120


def test_plain_attn_by_hand():
    values = np.zeros((2, 1, 2, 64, 128))
    values[1, 0, 0, 0, 0], values[1, 0, 1, 0], values[1, 0, 1, 1] = 4.0, 1.0, 3.0
    Q = np.zeros((1, 1, 128))
    Q[0, 0, 0] = np.log(3.0)
    O, lse, _, _ = ref.attn(Q, values, np.full((2, 1, 2), 0.5), np.array([[1]]), [2], sm_scale=0.5)
    assert np.allclose(O, (3 * 0.5 + 1.5) / 4) and np.allclose(lse, np.log(4.0))   # weights 3/4 and 1/4, values 0.5 and 1.5
