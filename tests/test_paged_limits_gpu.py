"""The paged 8-bit cache at the ends of what it accepts: the largest table, scales far apart or
no powers of two, what the status word says, and workspaces whose call gave up."""
import numpy as np
import pytest
import torch

import paged_utils as ref
from block_sparse_long_pool_gb300 import binding
from test_paged_gpu import BLK, D, DEV, F8, Attn, Cache, Plan, attn_case, i32, rows

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


# ---------------------------------------------------------------- append


def test_append_of_single_rows_is_the_same_in_every_call():
    """512 runs of one row, of which half make their page's scale grow, on equal caches: the old
    scale is read by all of a warp's lanes before one of them replaces it."""
    rng = np.random.default_rng(31)
    n, H = 512, 4
    first = None
    k, v = rows(rng, n, H, True)
    k = k * torch.as_tensor(2.0 ** rng.integers(-6, 7, n), device=DEV).to(torch.bfloat16)[:, None, None]
    slots = [p * BLK + int(r) for p, r in enumerate(rng.integers(1, BLK, n))]
    c = Cache(rng, n, H)
    was, old = c.pages.clone(), c.scale.clone()
    want = ref.append(*c.state()[:2], ref.f64(k), ref.f64(v), slots)
    grown = (want[1] > ref.f64(old)).mean()
    assert 0.2 < grown < 0.8
    t = i32(slots)
    for _ in range(50):
        c.pages.copy_(was)
        c.scale.copy_(old)
        binding.sparse_paged_append_f8(c.pages, c.scale, k, v, t, status=c.status)
        now = c.pages.view(torch.uint8).clone(), c.scale.clone()
        first = first or now
        assert torch.equal(now[0], first[0]) and torch.equal(now[1], first[1])
    c.check((want[0], want[1], None))


@pytest.mark.parametrize("n", [1, 2, 3, 40])
@pytest.mark.parametrize("old", [7.0, 0.3, 1.0 / 3, 3 * 2.0 ** -119, 1.9999998 * 2.0 ** 100, 5.0])
def test_append_to_pages_with_other_scales(n, old):
    """Pages whose scale is no power of two: rows are divided by it.  With a scale of 7, 175 is 25
    units, a tie that goes to 24, where 175 times the rounded 1 / 7 is above it.  Row by row
    every bf16 mantissa of e4m3's range, ties among them."""
    rng = np.random.default_rng(n)
    c = Cache(rng, 3, 2)
    c.scale.fill_(old)
    s = float(c.scale[0, 0, 0])
    x = rng.integers(128, 256, (n, 2, D)) * 2.0 ** rng.integers(-16, 1, (n, 2, D))   # bf16, up to 255 units
    x[:, :, ::3] = rng.integers(1, 29, x[:, :, ::3].shape)                          # whole numbers: ties at 17, 19, ...
    k = ref.bf16(x * s if old in (7.0, 5.0) else x * 2.0 ** np.floor(np.log2(s)), DEV)
    v = ref.bf16(-x * 2.0 ** np.floor(np.log2(s)), DEV)
    if old == 7.0:
        k[0, 0, 0] = 175.0
    slots = [BLK + 9 + i for i in range(n)]
    want = ref.append(*c.state()[:2], ref.f64(k), ref.f64(v), slots)
    assert (want[1] == s).all()   # no scale grows
    c.append(k, v, slots)
    c.check((want[0], want[1], None))
    if old == 7.0:
        assert float(c.pages[1, 0, 0, 9, 0]) == 24.0
    # a louder row: the scale grows to a power of two, and every row before is rounded again
    k[0, 1, 5] = 500 * s
    slots = [BLK + 9 + n]
    want = ref.append(*c.state()[:2], ref.f64(k[:1]), ref.f64(v[:1]), slots)
    assert want[1][1, 1, 0] > s
    c.append(k[:1], v[:1], slots)
    c.check((want[0], want[1], None))


def test_append_rounds_quotients_and_products_once():
    """Scales next to thirds and sevenths of powers of two, where x / scale lies within 2^-25 of a tie
    that it is not: rounded to fp32 first it would become one."""
    rng = np.random.default_rng(8)
    base = np.array([1 / 3, 1 / 7, 3 / 5, 5 / 3, 7 / 9, 9 / 11, 15 / 17, 1 / 13]) * 4
    near = np.float32(base)
    scales = np.concatenate([near, np.nextafter(near, np.float32(8)), np.nextafter(near, np.float32(0))])
    c = Cache(rng, len(scales), 1)
    c.scale[:] = torch.as_tensor(scales, device=DEV)[:, None, None]
    x = np.tile(np.arange(128, 256), (2 * len(scales), 1, 1)) * 0.25
    x[1::2] *= 4
    k, v = ref.bf16(x, DEV), ref.bf16(-x / 8, DEV)
    slots = [p * BLK + 3 + i for p in range(len(scales)) for i in (0, 1)]
    want = ref.append(*c.state()[:2], ref.f64(k), ref.f64(v), slots)
    c.append(k, v, slots)
    c.check((want[0], want[1], None))
    # grown by a row each: all that the page holds, times old scale / new scale
    k, v = ref.bf16(np.full((len(scales), 1, D), 3000.0), DEV), ref.bf16(np.full((len(scales), 1, D), 1500.0), DEV)
    slots = [p * BLK + 5 for p in range(len(scales))]
    want = ref.append(*c.state()[:2], ref.f64(k), ref.f64(v), slots)
    c.append(k, v, slots)
    c.check((want[0], want[1], None))


# ---------------------------------------------------------------- attention


def far_case(G, blocks, last, seed):
    """One request whose pages' scores and value scales differ by up to 2^230: what one loses by its
    softmax weight it gains by its values.  Scores in log2 units: block j's keys give about
    -level[j]; its value scale is 2^vs[j]."""
    rng = np.random.default_rng(seed)
    n = len(blocks) * BLK - (BLK - last)
    c = Cache(rng, len(blocks) + 1, 1)
    table = rng.permutation(len(blocks) + 1)[:len(blocks)][None].astype(np.int32)
    x = np.zeros((len(blocks) + 1, BLK, D), np.float32)
    x[:, :, 1:] = rng.standard_normal((len(blocks) + 1, BLK, D - 1))
    for j, (level, vs) in enumerate(blocks):
        x[table[0, j], :, 0] = level             # the query's first element is -1
        c.scale[int(table[0, j]), 0, 1] = 2.0 ** vs
    c.pages[:, 0, 0] = torch.as_tensor(x, device=DEV).to(F8)
    c.scale[:, 0, 0] = 1.0
    Q = rng.standard_normal((1, G, D)) * 0.125   # scores spread by a few log2 units
    Q[:, :, 0] = -1.0
    return c, table, [n], ref.bf16(Q, DEV)


@pytest.mark.parametrize("G", [1, 4, 8, 13, 16])
@pytest.mark.parametrize("last", [BLK, 37])
@pytest.mark.parametrize("blocks", [
    [(0, -118), (120, 110)], [(120, 110), (0, -118)],                 # 2^228 apart: the far block is O
    [(0, -118), (208, 110)], [(208, 110), (0, -118)],                 # its weights below 2^-126, its part 2^20 of O
    [(0, -100), (112, 6)], [(0, -60), (96, 40), (120, 64)],           # comparable parts of O
    [(0, -118), (224, 110), (104, -10)] * 2, [(52, 0), (0, -48), (104, 44)] * 20,
    # 8 blocks or fewer stay with one CTA: the same warp meets both kinds
    [(0, -118)] * 4 + [(120, 110)] * 4, [(120, 110)] * 3 + [(0, -118)] * 3, [(0, -118)] * 3 + [(208, 110)] * 3,
    [(208, 110)] * 4 + [(0, -118)] * 4, [(0, -100)] * 3 + [(112, 6)] * 3, [(0, -60)] * 3 + [(96, 40)] * 3,
    [(0, 110), (120, -118)]])
def test_attn_pages_whose_scales_are_far_apart_in_one_request(blocks, last, G):
    c, table, lens, Q = far_case(G, blocks, last, len(blocks) * 100 + G)
    a = Attn(1, G, 1)
    a.call(Q, c, i32(table), i32(lens), scale=float(np.log(2.0)))
    torch.cuda.synchronize()
    want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, lens, sm_scale=float(np.float32(np.log(2.0))))
    ref.assert_attn(a.O, a.lse, want, lens[0])
    assert a.status.item() == 0


# ---------------------------------------------------------------- what the status word says


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_tok", [1000, 4000])
def test_plan_with_an_unsound_input_and_a_refusal_reports_the_unsound_one(n_tok, in_place):
    """Each is found by another thread, CTA or launch; which one is reported does not depend on which
    of them is first."""
    B = 512
    table = np.zeros((B, 2), np.int32)
    table[:, 0] = np.arange(B)
    bad = binding.SPARSE_ERR_BAD_INDEX
    for at, refused in ((B - 1, 0), (0, B - 1), (300, 299)):
        for kind in ("length", "page"):
            lens = np.full(B, 60)
            new = np.ones(B, np.int64)
            new[refused] = 200                       # past its table
            t = table.copy()
            if kind == "length":
                lens[at] = -1
            else:
                t[at, 0] = B + 7                     # found by the row that is written there
            s = Plan(lens, t, np.full(B, -1), 0, n_tok)
            s.n_new.copy_(i32(new))
            for _ in range(20):
                s.seq_len.copy_(i32(lens))
                s.status.zero_()
                s.call(in_place)
                assert s.status.item() == bad, (kind, at)


def test_an_unsound_input_of_a_later_step_replaces_a_refusal():
    """A refusal is an ordinary end of a step; what follows it on the same word may not be."""
    s = Plan([60, 60], np.array([[0], [1]], np.int32), np.full(2, -1), 0, 8)
    for new, lens, want in (([9, 1], [60, 60], binding.SPARSE_ERR_NO_PAGES), ([1, 1], [60, 65], binding.SPARSE_ERR_BAD_INDEX),
                            ([9, 1], [60, 60], binding.SPARSE_ERR_BAD_INDEX)):
        s.n_new.copy_(i32(new))
        s.seq_len.copy_(i32(lens))
        s.call()
        assert s.status.item() == want


@pytest.mark.parametrize("G", [4, 16])
def test_attn_on_a_workspace_whose_call_gave_up(G):
    """The first word of the workspace as a call that gave up leaves it: every call reports it, over
    anything milder, until the workspace is zeroed."""
    rng = np.random.default_rng(G)
    lens = [3000, 100]
    c, table, Q = attn_case(rng, lens, 2, G)
    want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, lens)
    a = Attn(2, 2 * G, 2)
    a.ws[:4].view(torch.int32).fill_(1)
    for before, n in ((0, lens), (binding.SPARSE_ERR_BAD_INDEX, lens), (0, [3000, -1]), (0, [0, 0])):
        a.status.fill_(before)
        a.call(Q, c, i32(table), i32(n))
        assert a.status.item() == binding.SPARSE_ERR_TIMEOUT, n
    binding.sparse_paged_decode_attn_f8(Q, c.pages, c.scale, i32(table), i32(lens), a.O, a.ws)   # no status word
    a.ws.zero_()
    a.status.zero_()
    a.call(Q, c, i32(table), i32(lens))
    assert a.status.item() == 0
    ref.assert_attn(a.O, a.lse, want, 3000)
    assert not a.ws[:1 << 20].any()   # the counters and the word: zero after the call
