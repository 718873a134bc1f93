"""The paged 8-bit cache: page plan, append and decode attention against plain
implementations in 64 bits, and a run of them together with the Forecast selection."""
import numpy as np
import pytest
import torch

import paged_utils as ref
from block_sparse_long_pool_gb300 import binding

pytestmark = pytest.mark.gpu

BLK, D = 64, 128
DEV = "cuda"
F8 = torch.float8_e4m3fn


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def filled(n, v=-9):
    return torch.full((n,), v, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- page plan


class Plan:
    """Buffers of one batch's page plan, and the call."""

    def __init__(self, lens, table, free_pages, n_free, n_tok):
        B = len(lens)
        self.seq_len, self.table, self.free = i32(lens), i32(table), i32(free_pages)
        self.n_free, self.n_new = i32([n_free]), filled(B, 0)
        self.cu, self.start = filled(B + 1), filled(B)
        self.len_out, self.n_free_out = filled(B), filled(1)
        self.slot, self.req, self.pos = filled(n_tok), filled(n_tok), filled(n_tok)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(self, in_place=False, stream=None):
        binding.sparse_page_plan(self.seq_len, self.n_new, self.table, self.free, self.n_free, self.cu, self.start,
                                 self.seq_len if in_place else self.len_out, self.n_free if in_place else self.n_free_out,
                                 self.slot, self.req, self.pos, status=self.status, stream=stream)

    def check(self, want, in_place=False):
        torch.cuda.synchronize()
        got = dict(table=self.table, free=self.free, cu=self.cu, start=self.start, slot=self.slot, req=self.req,
                   pos=self.pos, len=self.seq_len if in_place else self.len_out)
        for name, t in got.items():
            assert np.array_equal(t.cpu().numpy(), np.asarray(want[name])), name
        assert (self.n_free if in_place else self.n_free_out).item() == want["n_free"]


def batch(rng, B, max_blocks, extra_pages, max_len=None):
    """Lengths, a table that holds their pages and a shuffled free list."""
    lens = [int(rng.integers(0, (max_len or max_blocks * BLK) + 1)) for _ in range(B)]
    held = sum(ref.nblk(n) for n in lens)
    perm = rng.permutation(held + extra_pages).astype(np.int32)
    table, at = np.full((B, max_blocks), -1, np.int32), 0
    for b, n in enumerate(lens):
        table[b, :ref.nblk(n)] = perm[at:at + ref.nblk(n)]
        at += ref.nblk(n)
    free = np.full(held + extra_pages, -1, np.int32)
    free[:extra_pages] = perm[held:]
    return lens, table, free, extra_pages


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,max_blocks,extra,n_tok,kind", [
    (1, 1, 1, 1, "decode"), (1, 3, 2, 200, "prompt"), (3, 5, 4, 3, "decode"), (33, 9, 40, 64, "mixed"),
    (129, 40, 700, 5000, "mixed"), (512, 17, 2000, 16384, "mixed"), (1025, 6, 1500, 1030, "decode"),
    (4096, 3, 5000, 8191, "mixed"), (7, 300, 2500, 70001, "prompt"), (64, 80, 3000, 131072, "prompt"),
    (20, 30, 11, 3000, "short"), (200, 30, 60, 9000, "short"), (40, 30, 0, 50, "decode")])
def test_page_plan(B, max_blocks, extra, n_tok, kind, in_place):
    rng = np.random.default_rng(B * 7919 + max_blocks)
    lens, table, free, n_free = batch(rng, B, max_blocks, extra, None if kind != "prompt" else 70)
    if kind == "decode":
        new = rng.integers(0, 2, B)
    elif kind == "prompt":
        new = rng.multinomial(n_tok - 1, np.ones(B) / B)
    else:
        new = np.where(rng.random(B) < 0.2, -1, rng.integers(0, 1 + max(1, 2 * n_tok // B), B))
        if kind == "mixed":
            new = np.where(rng.random(B) < 0.6, np.minimum(new, 1), new)
    want = ref.plan(lens, new, table, free, n_free, n_tok)
    s = Plan(lens, table, free, n_free, n_tok)
    s.n_new.copy_(i32(new))
    s.call(in_place)
    s.check(want, in_place)
    assert s.status.item() == (binding.SPARSE_ERR_NO_PAGES if want["refused"] else 0)
    live = want["slot"][want["slot"] >= 0]
    assert len(np.unique(live)) == len(live)


def test_page_plan_refuses_in_order_and_goes_on():
    # 4 pages free: request 0 takes 3, request 1 wants 2 (refused), request 2 wants 1 (refused:
    # the needs before it count), request 3 needs none, request 4 would not fit its table
    lens, table = [0, 64, 64, 10, 100], np.array([[-1] * 4, [4, -1, -1, -1], [5, -1, -1, -1], [6, -1, -1, -1],
                                                 [7, 8, -1, -1]], np.int32)
    free = np.array([0, 1, 2, 3, -1, -1, -1, -1, -1], np.int32)
    s = Plan(lens, table, free, 4, 1000)
    s.n_new.copy_(i32([192, 65, 1, 54, 157]))
    s.call()
    s.check(ref.plan(lens, [192, 65, 1, 54, 157], table, free, 4, 1000))
    assert s.start.tolist() == [0, -1, -1, 10, -1] and s.len_out.tolist() == [192, 64, 64, 64, 100]
    assert s.table[0].tolist() == [3, 2, 1, -1] and s.n_free_out.item() == 1
    assert s.status.item() == binding.SPARSE_ERR_NO_PAGES


def test_page_plan_rows_that_run_out():
    # 10 rows: the second request's rows end past them, the third has none left
    lens, table = [5, 5, 5], np.array([[0], [1], [2]], np.int32)
    s = Plan(lens, table, np.full(3, -1, np.int32), 0, 10)
    s.n_new.copy_(i32([6, 5, 1]))
    s.call()
    s.check(ref.plan(lens, [6, 5, 1], table, np.full(3, -1, np.int32), 0, 10))
    assert s.start.tolist() == [5, -1, -1] and s.cu.tolist() == [0, 6, 11, 12]


def test_page_plan_unsound_inputs_are_reported():
    table = np.array([[0, 1], [2, 3], [4, 99]], np.int32)
    # request 0: a length past its table; 1: ended with a negative length; 2: a page outside
    s = Plan([129, -5, 70], table, np.array([5, 6, -1, -1, -1, -1, -1], np.int32), 2, 8)
    s.n_new.copy_(i32([1, -1, 2]))
    s.call()
    torch.cuda.synchronize()
    assert s.status.item() == binding.SPARSE_ERR_BAD_INDEX
    assert s.start.tolist() == [-1, 0, 70] and s.len_out.tolist() == [129, 0, 72] and s.n_free_out.item() == 2
    assert s.slot.tolist() == [-1] * 8 and s.req.tolist() == [-1, 2, 2] + [-1] * 5
    # a free count past the list, and more pages returned than it holds
    s = Plan([64, 64], np.array([[0], [1]], np.int32), np.array([0, 1], np.int32), 5, 4)
    s.n_new.copy_(i32([-1, 0]))
    s.call()
    torch.cuda.synchronize()
    assert s.status.item() == binding.SPARSE_ERR_BAD_INDEX and s.n_free_out.item() == 2
    # new token counts whose sum passes 32 bits
    s = Plan([0, 0, 0], np.full((3, 1), -1, np.int32), np.array([0, 1], np.int32), 2, 4)
    s.n_new.copy_(i32([2 ** 31 - 1, 2 ** 31 - 1, 1]))
    s.call()
    torch.cuda.synchronize()
    assert s.cu.tolist() == [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1] and s.slot.tolist() == [-1] * 4
    assert s.start.tolist() == [-1, -1, -1] and s.status.item() == binding.SPARSE_ERR_NO_PAGES


def test_page_plan_captured_steps():
    """Decode steps of one captured graph, lengths and free count kept in place."""
    rng = np.random.default_rng(5)
    lens, table, free, n_free = batch(rng, 37, 12, 300, 500)
    s = Plan(lens, table, free, n_free, 40)
    s.n_new.fill_(1)
    s.call()   # outside the capture first: kernel attributes are set once
    s.table.copy_(i32(table))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call(in_place=True)
    for step in range(70):
        want = ref.plan(lens, [1] * 37, table, free, n_free, 40)
        g.replay()
        s.check(want, in_place=True)
        lens, table, free, n_free = want["len"].tolist(), want["table"], want["free"], want["n_free"]


# ---------------------------------------------------------------- append


class Cache:
    def __init__(self, rng, n_pages, H, B=1, N_cap=1):
        x = rng.standard_normal((n_pages, H, 2, BLK, D)) * 64
        self.pages = torch.as_tensor(x, dtype=torch.float32, device=DEV).clamp(-448, 448).to(F8)
        self.scale = torch.as_tensor(2.0 ** rng.integers(-9, -4, (n_pages, H, 2)), dtype=torch.float32, device=DEV)
        self.ktil = torch.as_tensor(rng.standard_normal((B, H, N_cap, D)), dtype=torch.float32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.H = H

    def state(self):
        return ref.f8_values(self.pages), ref.f64(self.scale), ref.f64(self.ktil)

    def append(self, k, v, slots, req=None, pos=None, stream=None):
        binding.sparse_paged_append_f8(self.pages, self.scale, k, v, i32(slots), None if req is None else self.ktil,
                                       None if req is None else i32(req), None if req is None else i32(pos),
                                       status=self.status, stream=stream)

    def check(self, want, mag=8.0):
        """mag: a bound of the keys' and means' absolute values."""
        torch.cuda.synchronize()
        values, scale, ktil = want
        assert np.array_equal(ref.f64(self.scale), scale)
        assert np.array_equal(ref.f8_values(self.pages), values, equal_nan=True)
        if ktil is not None:
            # up to 64 sums, a product and a quotient in fp32
            assert np.abs(ref.f64(self.ktil) - ktil).max() <= 66 * 2.0 ** -24 * mag


def rows(rng, T, H, strided, amp=1.0):
    wide = torch.as_tensor(rng.standard_normal((T, 3 * H * D)) * amp, dtype=torch.float32, device=DEV).clamp(-7.9, 7.9)
    wide = wide.to(torch.bfloat16)
    k, v = (wide[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in (1, 2))
    return (k, v) if strided else (k.contiguous(), v.contiguous())


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("H,lens,new", [
    (1, [0], [1]), (1, [63], [1]), (2, [64], [1]), (3, [17], [200]), (8, [5, 0, 64, 127, 1000], [1, 1, 1, 1, 1]),
    (8, [0, 61, 128, 7], [130, 3, 0, 64]), (2, [10] * 70, [1] * 70), (1, [0, 30, 0], [4000, 1, 777]), (16, [40], [90]),
    (4, [1, 62, 64, 129, 0, 0, 9], [64, 2, 65, 700, 1, 63, 301])])
def test_append(H, lens, new, strided):
    rng = np.random.default_rng(H * 1000 + sum(lens) + sum(new))
    B, pad = len(lens), 3
    N = max(ref.nblk(a + b) for a, b in zip(lens, new))
    table = rng.permutation(B * N + 2)[:B * N].reshape(B, N)
    slots, req, pos = [], [], []
    for b, (a, n) in enumerate(zip(lens, new)):
        for x in range(a, a + n):
            slots.append(int(table[b, x // BLK]) * BLK + x % BLK)
            req.append(b)
            pos.append(x)
    slots, req, pos = slots + [-1] * pad, req + [-1] * pad, pos + [-1] * pad
    c = Cache(rng, B * N + 2, H, B, N)
    k, v = rows(rng, len(slots), H, strided, amp=1.0 if sum(new) % 2 else 0.02)
    want = ref.append(*c.state()[:2], ref.f64(k), ref.f64(v), slots, c.state()[2], req, pos)
    c.append(k, v, slots, req, pos)
    c.check(want)
    assert c.status.item() == 0


@pytest.mark.parametrize("n_tok", [200, 420, 800, 1500])
def test_append_short_and_long_runs_side_by_side(n_tok):
    """64 heads, so that a CTA looks over 8, 16, 32 or 64 rows: runs of one row to whole pages
    in one window, rows without a slot between them, pages that held rows before."""
    rng = np.random.default_rng(n_tok)
    H, slots, req, pos, lens = 64, [], [], [], []
    while len(slots) < n_tok:
        new = int(rng.choice([1, 1, 1, 1, 2, 2, 3, 7, 40, 64, 90]))
        b, a = len(lens), int(rng.integers(0, 2 * BLK))
        for x in range(a, a + new):
            slots.append((3 * b + x // BLK - a // BLK) * BLK + x % BLK)
            req.append(b)
            pos.append(x)
        lens.append(a + new)
        if rng.random() < 0.2:
            slots, req, pos = slots + [-1], req + [-1], pos + [-1]
    B, N = len(lens), max(ref.nblk(n) for n in lens)
    c = Cache(rng, 3 * B, H, B, N)
    k, v = rows(rng, len(slots), H, True)
    want = ref.append(*c.state()[:2], ref.f64(k), ref.f64(v), slots, c.state()[2], req, pos)
    c.append(k, v, slots, req, pos)
    c.check(want)
    assert c.status.item() == 0


def test_append_row_by_row_gives_one_scale_and_the_pooled_keys():
    """64 calls of one row each: the scale grows, and rows rounded before are moved exactly."""
    rng = np.random.default_rng(3)
    c = Cache(rng, 2, 2, 1, 1)
    k, v = rows(rng, 64, 2, False)
    k = k * torch.logspace(-2, 2, 64, base=2.0, device=DEV).to(torch.bfloat16)[:, None, None]
    want = c.state()
    for t in range(64):
        want = ref.append(want[0], want[1], ref.f64(k[t:t + 1]), ref.f64(v[t:t + 1]), [64 + t], want[2], [0], [t])
        c.append(k[t:t + 1], v[t:t + 1], [64 + t], [0], [t])
        c.check(want, mag=100.0)   # 64 updates of a mean below 32, three roundings each
    assert np.array_equal(want[1][0], ref.f64(c.scale)[0])


@pytest.mark.parametrize("fill", ["zero", "tiny", "huge", "inf", "nan", "all_nan", "edge"])
def test_append_extreme_values(fill):
    rng = np.random.default_rng(11)
    c = Cache(rng, 3, 1)
    k, v = rows(rng, 40, 1, False)
    if fill == "zero":
        k.zero_()
    elif fill == "tiny":
        k.mul_(2.0 ** -126)
    elif fill == "huge":
        k.mul_(2.0 ** 124)
        k[3, 0, 5] = torch.finfo(torch.bfloat16).max
    elif fill == "inf":
        k[7, 0, 9], k[8, 0, 1], v[1, 0, 0] = float("inf"), float("-inf"), float("inf")
    elif fill == "nan":
        k[7, 0, 9], v[39, 0, 127] = float("nan"), float("nan")
    elif fill == "all_nan":
        k.fill_(float("nan"))
    else:
        k.fill_(0.0)
        k[0, 0, :4] = torch.tensor([448.0, -448.0, 450.0, 0.015625], device=DEV, dtype=torch.bfloat16)
    slots = [70 + i for i in range(40)]   # rows 6..45 of page 1: it holds rows already
    want = ref.append(*c.state()[:2], ref.f64(k), ref.f64(v), slots)
    c.append(k, v, slots)
    c.check((want[0], want[1], None))


def test_append_skips_pages_outside_and_reports_them():
    rng = np.random.default_rng(2)
    c = Cache(rng, 3, 2, 2, 2)
    k, v = rows(rng, 6, 2, False)
    slots, req, pos = [3 * BLK, 3 * BLK + 1, -1, 2 * BLK + 63, 0, 1], [0, 0, -1, 2, 1, 1], [0, 1, -1, 63, 64, 65]
    want = ref.append(*c.state()[:2], ref.f64(k), ref.f64(v), slots, c.state()[2], req, pos)
    c.append(k, v, slots, req, pos)
    c.check(want)
    assert c.status.item() == binding.SPARSE_ERR_BAD_INDEX


def test_append_far_pages():
    """Byte offsets past 32 bits."""
    n_pages, H = 36000, 8
    pages = torch.empty((n_pages, H, 2, BLK, D), dtype=torch.uint8, device=DEV).view(F8)
    scale = torch.ones((n_pages, H, 2), device=DEV)
    rng = np.random.default_rng(4)
    k, v = rows(rng, 70, H, False)
    slots = [(n_pages - 2) * BLK + i for i in range(70)]
    binding.sparse_paged_append_f8(pages, scale, k, v, i32(slots))
    zero = np.zeros((2, H, 2, BLK, D))
    want = ref.append(zero, np.ones((2, H, 2)), ref.f64(k), ref.f64(v), list(range(70)))
    got = ref.f8_values(pages[-2:])
    assert np.array_equal(got[0], want[0][0]) and np.array_equal(got[1, :, :, :6], want[0][1, :, :, :6])
    assert np.array_equal(ref.f64(scale[-2:]), want[1])


# ---------------------------------------------------------------- attention


def attn_case(rng, lens, H, G, extra_blocks=1, amp=1.0):
    B = len(lens)
    max_blocks = max(1, max(ref.nblk(n) for n in lens)) + extra_blocks
    n_pages = sum(ref.nblk(n) for n in lens) + 2
    c = Cache(rng, n_pages, H)
    perm = rng.permutation(n_pages)
    table, at = np.full((B, max_blocks), -1, np.int32), 0
    for b, n in enumerate(lens):
        table[b, :ref.nblk(n)] = perm[at:at + ref.nblk(n)]
        at += ref.nblk(n)
        if n % BLK:   # bytes of an earlier owner behind the last token, NaN among them
            c.pages.view(torch.uint8)[int(table[b, n // BLK]), :, :, n % BLK:] = torch.randint(
                0, 256, (H, 2, BLK - n % BLK, D), dtype=torch.uint8, device=DEV)
            c.pages.view(torch.uint8)[int(table[b, n // BLK]), :, :, n % BLK:, ::3] = 0x7f
    Q = torch.as_tensor(rng.standard_normal((B, H * G, D)) * amp, dtype=torch.float32, device=DEV).to(torch.bfloat16)
    return c, table, Q


class Attn:
    def __init__(self, B, H_q, H):
        self.O = torch.full((B, H_q, D), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((B, H_q), 7.0, device=DEV)
        self.ws = binding.paged_workspace(B, H_q, H)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(self, Q, c, table, lens, idx=None, count=None, scale=0.0, stream=None):
        binding.sparse_paged_decode_attn_f8(Q, c.pages, c.scale, table, lens, self.O, self.ws, blk_idx=idx, count=count,
                                            lse=self.lse, scale=scale, status=self.status, stream=stream)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 9, 16])
@pytest.mark.parametrize("H,lens", [
    (1, [1]), (2, [64]), (1, [65]), (3, [63, 0, 129]), (2, [1000, 1, 0, 64, 640]), (1, [0]), (1, [20000]),
    (4, [2049, 4096, 17]), (8, [300] * 40)])
def test_attn_all_blocks(H, lens, G):
    rng = np.random.default_rng(sum(lens) * 31 + G)
    c, table, Q = attn_case(rng, lens, H, G)
    a = Attn(len(lens), H * G, H)
    want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, lens)
    for _ in range(2):   # twice: the workspace's counters are back at zero
        a.O.fill_(7.0)
        a.call(Q, c, i32(table), i32(lens))
        torch.cuda.synchronize()
        ref.assert_attn(a.O, a.lse, want, max(lens))
    assert a.status.item() == 0


@pytest.mark.parametrize("G,H,lens,k", [(4, 2, [4096], 11), (8, 8, [9000, 70, 0, 12345], 19), (16, 1, [6400, 6401], 100),
                                        (1, 4, [700, 64, 65], 3), (7, 2, [2000] * 5, 1), (8, 3, [130], 6)])
def test_attn_selected_blocks(G, H, lens, k):
    rng = np.random.default_rng(k * 7 + G)
    c, table, Q = attn_case(rng, lens, H, G)
    B = len(lens)
    idx, count = np.full((B, H, k), -1, np.int32), np.zeros((B, H), np.int32)
    for b, n in enumerate(lens):
        for g in range(H):
            m = min(k, ref.nblk(n)) if g % 3 != 2 else min(k, ref.nblk(n)) // 2
            idx[b, g, :m] = np.sort(rng.permutation(ref.nblk(n))[:m])
            count[b, g] = m
    a = Attn(B, H * G, H)
    a.call(Q, c, i32(table), i32(lens), i32(idx), i32(count))
    torch.cuda.synchronize()
    want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, lens, idx, count)
    ref.assert_attn(a.O, a.lse, want, k * BLK)
    assert a.status.item() == 0


def test_attn_lists_and_tables_outside_are_skipped_and_reported():
    rng = np.random.default_rng(9)
    lens = [500, 500, 500, 500, 5000]
    c, table, Q = attn_case(rng, lens[:4] + [500], 2, 4)
    max_blocks = table.shape[1]
    idx = np.tile(np.arange(6, dtype=np.int32), (5, 2, 1))
    count = np.full((5, 2), 6, np.int32)
    want_status = binding.SPARSE_ERR_BAD_INDEX
    idx[0, 0, 2] = -3
    idx[0, 1, 5] = max_blocks
    idx[1, 0, 5] = max_blocks - 1      # past the length: nothing, not an error
    table[2, 3] = c.pages.shape[0]
    table[3, 1] = -1
    count[3, 1] = 9                    # clamped to 6
    a = Attn(5, 8, 2)
    a.call(Q, c, i32(table), i32(lens), i32(idx), i32(count))   # request 4: a length past its table
    torch.cuda.synchronize()
    want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, lens, idx, count)
    ref.assert_attn(a.O, a.lse, want, 384)
    assert a.status.item() == want_status
    # a negative count and a negative length: no tokens
    a.status.zero_()
    count[0] = -1
    a.call(Q, c, i32(table), i32([500, -1, 500, 500, 500]), i32(idx), i32(count))
    torch.cuda.synchronize()
    assert a.status.item() == want_status and (a.O[:2] == 0).all() and torch.isinf(a.lse[:2]).all()


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("length", [-1, 4 * BLK + 1])
def test_attn_a_length_outside_its_table_is_reported(selected, length):
    rng = np.random.default_rng(10)
    c, table, Q = attn_case(rng, [200, 250], 2, 2, extra_blocks=0)
    a = Attn(2, 4, 2)
    idx, count = i32(np.tile(np.arange(4), (2, 2, 1))), i32(np.full((2, 2), 4))
    a.call(Q, c, i32(table), i32([200, length]), *((idx, count) if selected else ()))
    torch.cuda.synchronize()
    assert a.status.item() == binding.SPARSE_ERR_BAD_INDEX
    want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, [200, 0])
    ref.assert_attn(a.O[:1], a.lse[:1], [x[:1] for x in want], 256)
    if length < 0:
        assert (a.O[1] == 0).all() and torch.isinf(a.lse[1]).all()


def test_attn_values_of_tiny_and_huge_pages():
    """Value scales at the ends of what the append writes: outputs near fp32's limits."""
    rng = np.random.default_rng(14)
    lens = [500, 500]
    c, table, Q = attn_case(rng, lens, 1, 8)
    used = torch.as_tensor(table[0][table[0] >= 0].astype(np.int64), device=DEV)
    c.scale[:, :, 1] = 2.0 ** 110
    c.scale[used, :, 1] = 2.0 ** -118
    a = Attn(2, 8, 1)
    a.call(Q, c, i32(table), i32(lens))
    torch.cuda.synchronize()
    want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, lens)
    for b in range(2):
        ref.assert_attn(a.O[b:b + 1], a.lse[b:b + 1], [x[b:b + 1] for x in want], 500)


def test_attn_scale_and_large_scores():
    """Scores of several hundred, a scale of the caller's, scales of very different pages."""
    rng = np.random.default_rng(21)
    lens = [700, 3000]
    c, table, Q = attn_case(rng, lens, 2, 8, amp=20.0)
    c.scale[:] = torch.as_tensor(2.0 ** rng.integers(-40, 10, tuple(c.scale.shape)), dtype=torch.float32, device=DEV)
    c.scale[:, :, 0] = torch.as_tensor(rng.uniform(0.004, 0.03, tuple(c.scale.shape[:2])), dtype=torch.float32, device=DEV)
    a = Attn(2, 16, 2)
    a.call(Q, c, i32(table), i32(lens), scale=0.25)
    torch.cuda.synchronize()
    want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, lens, sm_scale=0.25)
    ref.assert_attn(a.O, a.lse, want, max(lens))


def test_attn_query_rows_of_any_size():
    """bf16 queries far outside half precision's range, with keys that bring the scores back."""
    rng = np.random.default_rng(22)
    c, table, Q = attn_case(rng, [300], 1, 8)
    mul = torch.tensor([2.0 ** e for e in (100, 60, 17, 0, -14, -30, -60, -100)], device=DEV).to(torch.bfloat16)
    Q = Q * mul[None, :, None]
    Q[0, 3] = 0
    for e in (100, 17, 0, -30, -100):
        c.scale[:, :, 0] = 2.0 ** (-6 - e)
        a = Attn(1, 8, 1)
        rows_ok = [i for i, x in enumerate((100, 60, 17, 0, -14, -30, -60, -100)) if x <= e + 4]
        a.call(Q, c, i32(table), i32([300]))
        torch.cuda.synchronize()
        want = ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, [300])
        ref.assert_attn(a.O[:, rows_ok], a.lse[:, rows_ok], [x[:, rows_ok] for x in want], 300, f"2^{e}")


def test_attn_far_pages():
    """Byte offsets past 32 bits."""
    n_pages, H, G = 36000, 8, 4
    small = Cache(np.random.default_rng(8), 4, H)
    pages = torch.empty((n_pages, H, 2, BLK, D), dtype=torch.uint8, device=DEV).view(F8)
    scale = torch.ones((n_pages, H, 2), device=DEV)
    pages.view(torch.uint8)[-4:] = small.pages.view(torch.uint8)
    scale[-4:] = small.scale
    Q = torch.randn((1, H * G, D), device=DEV).to(torch.bfloat16)
    a = Attn(1, H * G, H)
    binding.sparse_paged_decode_attn_f8(Q, pages, scale, i32([[n_pages - 1, n_pages - 3, n_pages - 4]]), i32([170]), a.O,
                                        a.ws, lse=a.lse)
    torch.cuda.synchronize()
    want = ref.attn(ref.f64(Q), ref.f8_values(small.pages), ref.f64(small.scale), np.array([[3, 1, 0]]), [170])
    ref.assert_attn(a.O, a.lse, want, 170)


def test_attn_is_repeatable_and_runs_on_another_stream():
    rng = np.random.default_rng(13)
    lens = [9000, 100, 31000]
    c, table, Q = attn_case(rng, lens, 4, 8)
    t, n = i32(table), i32(lens)
    a, other = Attn(3, 32, 4), Attn(3, 32, 4)
    a.call(Q, c, t, n)
    torch.cuda.synchronize()
    first = a.O.clone(), a.lse.clone()
    side = torch.cuda.Stream()
    for _ in range(20):
        a.call(Q, c, t, n)
        other.call(Q, c, t, n, stream=side)   # two calls at once, each with its own workspace
    torch.cuda.synchronize()
    for x in (a, other):
        assert torch.equal(x.O, first[0]) and torch.equal(x.lse, first[1])


def test_attn_calls_of_different_sizes_share_a_workspace():
    rng = np.random.default_rng(41)
    shared = Attn(3, 48, 3)   # the largest workspace: more than 8 rows a pair
    for lens, H, G in (([9000, 1, 700], 3, 16), ([20000], 1, 4), ([300] * 3, 2, 8), ([5000, 4000], 2, 16), ([40000], 2, 1),
                       ([9000, 1, 700], 3, 16)):
        c, table, Q = attn_case(rng, lens, H, G)
        a = Attn(len(lens), H * G, H)
        a.ws = shared.ws
        a.call(Q, c, i32(table), i32(lens))
        torch.cuda.synchronize()
        ref.assert_attn(a.O, a.lse, ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), table, lens), max(lens))
        assert a.status.item() == 0


def test_attn_lists_of_nothing():
    """Every listed block outside, or past the length: no tokens, but a row that is written."""
    rng = np.random.default_rng(43)
    c, table, Q = attn_case(rng, [100, 100, 5000], 2, 5, extra_blocks=0)
    idx = np.tile(np.arange(70, dtype=np.int32), (3, 2, 1))
    idx[0], idx[1] = -1, np.arange(2, 72)   # request 1: past its length, or (past 78 blocks) outside
    a = Attn(3, 10, 2)
    a.call(Q, c, i32(table), i32([100, 100, 0]), i32(idx), i32(np.full((3, 2), 70)))
    torch.cuda.synchronize()
    assert (a.O == 0).all() and torch.isinf(a.lse).all() and (a.lse < 0).all()
    assert a.status.item() == binding.SPARSE_ERR_BAD_INDEX


def test_attn_a_query_of_nan_stays_in_its_row():
    rng = np.random.default_rng(44)
    for G in (4, 16):
        c, table, Q = attn_case(rng, [700], 2, G)
        a = Attn(1, 2 * G, 2)
        Q[0, 2, 17] = float("nan")
        a.call(Q, c, i32(table), i32([700]))
        torch.cuda.synchronize()
        assert torch.isnan(a.O[0, 2]).all()
        keep = [r for r in range(2 * G) if r != 2]
        want = ref.attn(ref.f64(Q[:, keep]).reshape(1, -1, D), ref.f8_values(c.pages)[:, :1], ref.f64(c.scale)[:, :1], table, [700])
        ref.assert_attn(a.O[:, keep[:G - 1]], a.lse[:, keep[:G - 1]], [x[:, :G - 1] for x in want], 700)


def test_attn_captured_with_lengths_that_grow():
    """One captured call, replayed as the lengths grow over page ends and a request appears,
    with eager calls on another workspace between."""
    rng = np.random.default_rng(45)
    c, table, Q = attn_case(rng, [2600, 130, 64], 2, 6)
    a, eager = Attn(3, 12, 2), Attn(3, 12, 2)
    t, lens = i32(table), i32([2500, 60, 0])
    a.call(Q, c, t, lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(Q, c, t, lens)
    pages = ref.f8_values(c.pages)
    for now in ([2500, 60, 0], [2560, 64, 1], [2561, 65, 63], [2600, 130, 64], [0, 0, 0], [1, 129, 2]):
        lens.copy_(i32(now))
        g.replay()
        eager.call(Q, c, t, lens)
        torch.cuda.synchronize()
        want = ref.attn(ref.f64(Q), pages, ref.f64(c.scale), table, now)
        for x in (a, eager):
            ref.assert_attn(x.O, x.lse, want, 2600, str(now))


def test_attn_many_calls_of_a_full_grid():
    """Every SM busy, ranges that begin and end inside a pair's list: the same bits each time,
    equal to the plain implementation for a few pairs."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    B, H, G, k, max_blocks, n_pages = 8, 8, 8, 67, 300, 900
    pages = (torch.randn((n_pages, H, 2, BLK, D), generator=g, device=DEV) * 64).clamp(-448, 448).to(F8)
    scale = torch.full((n_pages, H, 2), 2.0 ** -6, device=DEV)
    table = torch.randint(0, n_pages, (B, max_blocks), generator=g, device=DEV, dtype=torch.int32)
    lens = i32([max_blocks * BLK - 7 * b for b in range(B)])
    idx = torch.rand((B, H, max_blocks), generator=g, device=DEV).argsort(2)[:, :, :k].sort(2).values.to(torch.int32)
    count = torch.randint(k // 2, k + 1, (B, H), generator=g, device=DEV, dtype=torch.int32)
    Q = torch.randn((B, H * G, D), generator=g, device=DEV).to(torch.bfloat16)
    a = Attn(B, H * G, H)
    for i in range(100):
        binding.sparse_paged_decode_attn_f8(Q, pages, scale, table, lens, a.O, a.ws, blk_idx=idx, count=count, lse=a.lse,
                                            status=a.status)
        if i == 0:
            first = a.O.clone(), a.lse.clone()
    torch.cuda.synchronize()
    assert a.status.item() == 0 and torch.equal(a.O, first[0]) and torch.equal(a.lse, first[1])
    for b in (0, 5):
        rows = slice(b, b + 1)
        want = ref.attn(ref.f64(Q[rows]), ref.f8_values(pages), ref.f64(scale), table[rows].cpu().numpy(),
                        lens[rows].cpu().numpy(), idx[rows].cpu().numpy(), count[rows].cpu().numpy())
        ref.assert_attn(a.O[rows], a.lse[rows], want, k * BLK)


@pytest.mark.parametrize("G", [1, 4, 5, 8, 9, 16])
def test_attn_many_short_parts_of_a_full_grid(G):
    """1200 pairs of 0 to 20 blocks, so that a CTA ends several parts of its own and shares
    the first and the last: the same bits each time, equal to the plain implementation."""
    rng = np.random.default_rng(G)
    B, H, max_blocks, n_pages = 150, 8, 20, 500
    g = torch.Generator(device=DEV)
    g.manual_seed(G)
    pages = (torch.randn((n_pages, H, 2, BLK, D), generator=g, device=DEV) * 64).clamp(-448, 448).to(F8)
    scale = torch.exp2(torch.randint(-8, -4, (n_pages, H, 2), generator=g, device=DEV).float())
    table = torch.randint(0, n_pages, (B, max_blocks), generator=g, device=DEV, dtype=torch.int32)
    lens = rng.integers(0, max_blocks * BLK + 1, B)
    lens[rng.permutation(B)[:60]] = rng.integers(0, 3 * BLK, 60)
    t_lens = i32(lens.tolist())
    Q = torch.randn((B, H * G, D), generator=g, device=DEV).to(torch.bfloat16)
    a = Attn(B, H * G, H)
    for i in range(60):
        binding.sparse_paged_decode_attn_f8(Q, pages, scale, table, t_lens, a.O, a.ws, lse=a.lse, status=a.status)
        if i == 0:
            first = a.O.clone(), a.lse.clone()
    torch.cuda.synchronize()
    assert a.status.item() == 0 and torch.equal(a.O, first[0]) and torch.equal(a.lse, first[1])
    values, scales = ref.f8_values(pages), ref.f64(scale)
    for b in (0, 1, 74, 75, 148, 149, int(lens.argmax()), int(lens.argmin())):
        rows = slice(b, b + 1)
        want = ref.attn(ref.f64(Q[rows]), values, scales, table[rows].cpu().numpy(), lens[rows])
        ref.assert_attn(a.O[rows], a.lse[rows], want, max_blocks * BLK)


# ---------------------------------------------------------------- refusals of the binding


def test_binding_refusals():
    s = Plan([1, 2], np.full((2, 3), 0, np.int32), np.arange(6), 6, 4)
    for name, bad, error in (("seq_len", s.seq_len.long(), TypeError), ("n_new", filled(3, 0), ValueError),
                             ("table", s.table.t(), ValueError), ("slot", s.slot.cpu(), ValueError),
                             ("status", torch.zeros(2, dtype=torch.int32, device=DEV), ValueError), ("cu", filled(2), ValueError),
                             ("free", None, TypeError)):
        keep = getattr(s, name)
        setattr(s, name, bad)
        with pytest.raises(error):
            s.call()
        setattr(s, name, keep)
    c = Cache(np.random.default_rng(1), 2, 2, 1, 1)
    k, v = rows(np.random.default_rng(1), 3, 2, True)
    wide = torch.zeros((3, 2, 2 * D), dtype=torch.bfloat16, device=DEV)
    for bad, error in ((k.float(), TypeError), (k[:2], ValueError), (k.transpose(0, 1).contiguous().transpose(0, 1), ValueError),
                       (wide[:, :, ::2], ValueError), (wide[:, :, :D], ValueError), (None, TypeError), (k.cpu(), ValueError)):
        with pytest.raises(error):
            c.append(bad, v, [0, 1, 2])
        with pytest.raises(error):
            c.append(k, bad, [0, 1, 2])
    with pytest.raises(ValueError, match="tok_req"):
        binding.sparse_paged_append_f8(c.pages, c.scale, k, v, i32([0, 1, 2]), c.ktil)
    with pytest.raises(TypeError):
        binding.sparse_paged_append_f8(c.pages.view(torch.uint8), c.scale, k, v, i32([0, 1, 2]))
    with pytest.raises(binding.SparsePoolError, match="strides"):   # rows that overlap
        flat = torch.zeros(3 * 256, dtype=torch.bfloat16, device=DEV)
        c.append(flat.as_strided((3, 2, D), (128, 128, 1)), v, [0, 1, 2])
    a = Attn(1, 8, 2)
    Q, t, n = torch.zeros((1, 8, D), dtype=torch.bfloat16, device=DEV), i32([[0]]), i32([5])
    with pytest.raises(binding.SparsePoolError, match="workspace"):
        binding.sparse_paged_decode_attn_f8(Q, c.pages, c.scale, t, n, a.O, a.ws[:4096])
    with pytest.raises(ValueError, match="count"):
        binding.sparse_paged_decode_attn_f8(Q, c.pages, c.scale, t, n, a.O, a.ws, blk_idx=i32([[[0], [0]]]))
    for bad in ({"Q": Q.float()}, {"Q": Q[:, :7]}, {"seq_len": n[:0]}, {"O": a.O.transpose(1, 2)}, {"lse": a.lse[:, :4]},
                {"block_table": t.long()}, {"workspace": a.ws.cpu()}, {"kv_scale": c.scale.half()}):
        args = {**dict(Q=Q, kv_pages=c.pages, kv_scale=c.scale, block_table=t, seq_len=n, O=a.O, workspace=a.ws), **bad}
        with pytest.raises((TypeError, ValueError)):
            binding.sparse_paged_decode_attn_f8(**args)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_a_serving_batch(graph):
    """Prompts, decode steps, an ended request and a new one in its place: plan, append,
    Forecast selection and attention, each against the plain implementation on the state
    that the calls left."""
    rng = np.random.default_rng(77)
    B, H, G, n_pages, max_blocks, k_tot = 4, 2, 4, 64, 16, 6
    plan = Plan([0] * B, np.full((B, max_blocks), -1, np.int32), rng.permutation(n_pages), n_pages, 700)
    one = Plan([0] * B, np.full((B, max_blocks), -1, np.int32), rng.permutation(n_pages), n_pages, 8)
    for name in ("seq_len", "table", "free", "n_free"):   # the decode plan works on the same batch
        setattr(one, name, getattr(plan, name))
    c = Cache(rng, n_pages, H, B, max_blocks)
    idx, count = torch.empty((B, H, k_tot), dtype=torch.int32, device=DEV), torch.empty((B, H), dtype=torch.int32, device=DEV)
    a = Attn(B, H * G, H)
    rows_k, rows_v = (torch.zeros((8, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    Q, F = torch.zeros((B, H * G, D), dtype=torch.bfloat16, device=DEV), torch.zeros((B, H, D), dtype=torch.bfloat16, device=DEV)

    def step(p, k, v):
        p.call(in_place=True)
        binding.sparse_paged_append_f8(c.pages, c.scale, k, v, p.slot, c.ktil, p.req, p.pos, status=c.status)
        binding.sparse_select_topk(F, c.ktil, p.seq_len, 1, 2, 3, idx, count, status=c.status)
        a.call(Q, c, p.table, p.seq_len, idx, count)

    def check(p, k, v, before, plan_before, new):
        torch.cuda.synchronize()
        want = ref.plan(*plan_before[:1], new, *plan_before[1:], p.slot.numel())
        p.check(want, in_place=True)
        after = ref.append(before[0], before[1], ref.f64(k), ref.f64(v), want["slot"], before[2], want["req"], want["pos"])
        c.check(after)
        n, ids = count.cpu().numpy(), idx.cpu().numpy()
        for b in range(B):
            nb = ref.nblk(int(want["len"][b]))
            assert (n[b] == min(nb, 6)).all()
            for g in range(H):
                mine = [j for j in ids[b, g] if j >= 0]
                assert set(range(min(1, nb))) | set(range(max(0, nb - 2), nb)) <= set(mine)
        ref.assert_attn(a.O, a.lse, ref.attn(ref.f64(Q), ref.f8_values(c.pages), ref.f64(c.scale), want["table"], want["len"],
                                             ids, n), 6 * BLK)

    def now(p):
        return (p.seq_len.tolist(), p.table.cpu().numpy(), p.free.cpu().numpy(), p.n_free.item())

    def values():
        Q.copy_(torch.as_tensor(rng.standard_normal(tuple(Q.shape))))
        F.copy_(torch.as_tensor(rng.standard_normal(tuple(F.shape))))

    new = [300, 64, 0, 333]
    plan.n_new.copy_(i32(new))
    k, v = rows(rng, 700, H, True)
    values()
    before, pb = c.state(), now(plan)
    step(plan, k, v)
    check(plan, k, v, before, pb, new)
    g = None
    if graph:
        # a captured decode step is replayed on buffers whose contents change; the calls ran
        # once before the capture
        g = torch.cuda.CUDAGraph()
        one.n_new.zero_()
        step(one, rows_k, rows_v)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            step(one, rows_k, rows_v)
    for i in range(6):
        new = [1, 1, 0, 1]
        if i == 2:
            new = [1, 1, 0, -1]        # request 3 ends
        elif i > 2:
            new = [1, 1, 2 if i == 4 else 0, 1]
        one.n_new.copy_(i32(new))
        k, v = rows(rng, 8, H, False)
        rows_k.copy_(k)
        rows_v.copy_(v)
        values()
        before, pb = c.state(), now(one)
        if g is not None:
            g.replay()
        else:
            step(one, rows_k, rows_v)
        check(one, rows_k, rows_v, before, pb, new)
    assert plan.seq_len.tolist() == [306, 70, 2, 3]
    assert c.status.item() == 0 and a.status.item() == 0 and one.status.item() == 0
