"""Plain implementations, in 64 bits, of chunk attention, rotary positions, forks and copies."""
from __future__ import annotations

import numpy as np
import torch

BLK, D = 64, 128


def nblk(n):
    return -(-n // BLK)


class Chunk:
    """A paged cache and a step's new rows, drawn from a seed."""

    def __init__(self, start, new, H_kv, G, seed=0, pad=0, first=0, strided=False, device="cuda", exps=(-7, -5), q_mag=1.0,
                 extra_blocks=3):
        g = torch.Generator().manual_seed(seed)
        B, H_q = len(start), H_kv * G
        self.first = first
        lens = [s + n if s >= 0 else 0 for s, n in zip(start, new)]
        self.max_blocks = max(1, max(nblk(n) for n in lens)) + extra_blocks
        self.n_pages = sum(nblk(n) for n in lens) + 5
        perm = torch.randperm(self.n_pages, generator=g).tolist()
        table = np.full((B, self.max_blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(lens):
            table[b, : nblk(n)] = perm[at : at + nblk(n)]
            at += nblk(n)
        pages = (torch.randn((self.n_pages, H_kv, 2, BLK, D), generator=g) * 80).clamp(-448, 448).to(torch.float8_e4m3fn)
        for b, n in enumerate(lens):   # any bytes behind the last token
            if n % BLK:
                pages[int(table[b, n // BLK]), :, :, n % BLK:] = float("nan")
        scale = torch.exp2(torch.randint(exps[0], exps[1], (self.n_pages, H_kv, 2), generator=g).float())
        n_tok = first + sum(new) + pad
        width = (H_q + 2 * H_kv if strided else H_q) * D
        q = (torch.randn((n_tok, width), generator=g) * q_mag).to(torch.bfloat16)
        self.B, self.H_kv, self.G, self.H_q, self.n_tok, self.lens = B, H_kv, G, H_q, n_tok, lens
        self.start_list, self.new_list = list(start), list(new)
        i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=device)
        self.table, self.pages, self.scale = i32(table), pages.to(device), scale.to(device)
        self.Q = q.to(device)[:, : H_q * D].view(n_tok, H_q, D)
        self.cu, self.start = i32(np.concatenate([[0], np.cumsum(new)]) + first), i32(start)
        self.O = torch.full((n_tok, H_q, D), 7.0, dtype=torch.bfloat16, device=device)
        self.lse = torch.full((n_tok, H_q), 7.0, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def call(self, workspace, **kw):
        from block_sparse_long_pool_gb300 import binding
        kw = {"lse": self.lse, "status": self.status, **kw}
        binding.sparse_paged_chunk_attn_f8(self.Q, self.pages, self.scale, self.table, self.cu, self.start, self.O, workspace, **kw)

    def expected(self, scale=D ** -0.5):
        """O, lse, and a bound of O's and of lse's error for each element, in 64 bits."""
        dev = self.pages.device
        O = torch.full((self.n_tok, self.H_q, D), 7.0, dtype=torch.float64, device=dev)
        lse = torch.full((self.n_tok, self.H_q), 7.0, dtype=torch.float64, device=dev)
        tol, tol_l = torch.zeros_like(O), torch.zeros_like(lse)
        cap = self.max_blocks * BLK
        row = self.first
        for b, (s, n) in enumerate(zip(self.start.tolist(), self.new_list)):
            r = slice(row, row + n)
            row += n
            if s < 0 or n == 0:
                O[r], lse[r] = 0.0, float("-inf")
                continue
            end = min(s + n, cap)
            page = self.table[b, : nblk(end)].long()
            ok = (page >= 0) & (page < self.n_pages)
            page = page.clamp(0, self.n_pages - 1)
            kv = self.pages[page].double() * self.scale[page].double()[..., None, None]
            kv = kv.permute(2, 1, 0, 3, 4).reshape(2, self.H_kv, -1, D)[:, :, :end]
            ok = ok.repeat_interleave(BLK)[:end]
            q = self.Q[r].double().view(n, self.H_kv, self.G, D).permute(1, 2, 0, 3)
            sc = torch.einsum("hgnd,htd->hgnt", q, kv[0]) * scale
            sabs = torch.einsum("hgnd,htd->hgnt", q.abs(), kv[0].abs().nan_to_num()) * abs(scale)
            see = (torch.arange(end, device=dev)[None] <= torch.arange(s, s + n, device=dev)[:, None]) & ok[None]
            sc = torch.where(see, sc, float("-inf"))
            top = sc.nan_to_num(nan=0.0).amax(-1, keepdim=True)
            p = torch.exp(sc - torch.where(top.isinf(), 0.0, top))
            total = p.sum(-1, keepdim=True)
            w = p / torch.where(total > 0, total, 1.0)
            v = torch.where(ok[:, None], kv[1], 0.0)
            # a value that a row does not see adds nothing, whatever it is
            o = torch.einsum("hgnt,htd->hgnd", w, v.nan_to_num())
            bad = torch.einsum("nt,htd->hnd", see.double(), v.isnan().double()) > 0
            o = torch.where(bad[:, None], float("nan"), o)
            o = torch.where(total.isnan(), float("nan"), o)
            size = torch.einsum("hgnt,htd->hgnd", w.nan_to_num(), v.nan_to_num().abs())
            # scores: fp32 sums of 128 exact products, one more product, an exponent in fp32 and 2^x (2^-22)
            ds = torch.where(see, sabs, 0.0).amax(-1, keepdim=True) * 132 * 2.0 ** -24 + 2.0 ** -22
            # queries in two e4m3 terms: the row's largest is scaled into (224, 448], each element is off by half of
            # e4m3's least step at most (2^-10; its first term leaves a rest of 4 bits where that step allows), so
            # by 2^-10 / 224 < 2^-17 of the largest, times the keys' sizes
            ksum = torch.where(ok[None, :], kv[0].abs().nan_to_num().sum(-1), 0.0).amax(-1)[:, None, None, None]
            ds = ds + q.abs().amax(-1, keepdim=True) * ksum * abs(scale) * 2.0 ** -17
            ds = ds + (sc.abs().where(see, torch.zeros_like(sc)).nan_to_num().amax(-1, keepdim=True) * 1.4427 + 16) * 2.0 ** -23
            # weights in f16 (2^-11, below 2^-14 of the best steps of 2^-24), fp32 sums over the steps; O in bf16
            t = o.nan_to_num().abs() * 2.0 ** -8 + size * (2.0 ** -11 + 2 * ds + 2.0 ** -18) * (1 + 2.0 ** -8)
            vmax = v.nan_to_num().abs().amax((1, 2))[:, None, None, None]
            t = t + 2.0 ** -25 * vmax * (w.nan_to_num() > 0).sum(-1, keepdim=True) / total.nan_to_num(nan=1.0).clamp(min=1.0)
            l = (top + torch.log(total))[..., 0]
            O[r] = o.permute(2, 0, 1, 3).reshape(n, self.H_q, D)
            tol[r] = t.permute(2, 0, 1, 3).reshape(n, self.H_q, D)
            lse[r] = l.permute(2, 0, 1).reshape(n, self.H_q)
            tol_l[r] = (2 * ds[..., 0] + 2.0 ** -18 + l.nan_to_num(neginf=0.0).abs() * 2.0 ** -22).permute(2, 0, 1).reshape(n, self.H_q)
        return O, lse, tol, tol_l

    def check(self, scale=D ** -0.5, status=0):
        torch.cuda.synchronize()
        assert self.status.item() == status
        O, lse, tol, tol_l = self.expected(scale)
        got = self.O.double()
        assert torch.equal(got.isnan(), O.isnan())
        err = (got - O).abs().nan_to_num()
        assert (err <= tol).all(), f"O off by {(err / tol.clamp(min=1e-30)).max().item():.3g} bounds"
        assert torch.equal(self.lse.isinf(), lse.isinf()) and torch.equal(self.lse.isnan(), lse.isnan())
        err = torch.where(lse.isfinite(), (self.lse.double() - lse).abs(), 0.0)
        assert (err <= tol_l).all(), f"lse off by {err.max().item():.3g}"


def rope(x, pos, inv_freq, interleaved, factor):
    """fp64: rows [n][H][128] turned; rows without a position are zero."""
    y = x.double().clone()
    half = inv_freq.numel()
    ang = pos.double()[:, None] * inv_freq
    c, s = torch.cos(ang)[:, None] * factor, torch.sin(ang)[:, None] * factor
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    xa, xb = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    size = x.double().abs()
    size[..., a] = size[..., b] = (xa.abs() + xb.abs()) * abs(factor)
    return torch.where((pos >= 0)[:, None, None], y, 0.0), size


def fork(src, seq_len, table, extra, free_pages, n_free, fork_len=None):
    """Request by request; numpy arrays, inputs unchanged."""
    B = len(src)
    table, extra, lens = table.copy(), extra.copy(), list(seq_len)
    free, tail = list(free_pages[:n_free]), list(free_pages[n_free:])
    gone = [b for b in range(B) if src[b] != b]
    left = {}
    for b in gone:
        for j in range(nblk(lens[b])):
            p = int(table[b, j])
            left[p] = left.get(p, int(extra[p]) + 1) - 1
    last = {int(table[b, j]): b for b in gone for j in range(nblk(lens[b]))}
    for b in gone:
        for j in range(nblk(lens[b])):
            p = int(table[b, j])
            if left[p] == 0 and last[p] == b:
                free.append(p)
    for p, n in left.items():
        extra[p] = max(n - 1, 0)
    F = len(free)
    pages_out = np.array((free + tail[F - n_free:])[: len(free_pages)], np.int32)
    copy_src, copy_dst = np.full(B, -1, np.int32), np.full(B, -1, np.int32)
    wanted = refused = 0
    new_len = list(lens)
    for b in gone:
        s = src[b]
        new_len[b] = 0
        if s < 0:
            continue
        n = lens[s]
        if fork_len is not None and 0 <= fork_len[b] < n:
            n = fork_len[b] // BLK * BLK
        if n % BLK:
            wanted += 1
            if wanted > F:
                refused += 1
                continue
            copy_src[b], copy_dst[b] = table[s, n // BLK], free[F - wanted]
            table[b, n // BLK] = free[F - wanted]
        for j in range(n // BLK):
            table[b, j] = table[s, j]
            extra[table[s, j]] += 1
        new_len[b] = n
    return dict(table=table, extra=extra, free=pages_out, n_free=F - min(wanted, F), len=np.array(new_len, np.int32), copy_src=copy_src,
                copy_dst=copy_dst, refused=refused)
