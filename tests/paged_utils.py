"""Plain implementations, in 64 bits, of the paged 8-bit cache's three calls."""
from __future__ import annotations

import numpy as np
import torch

BLK, D = 64, 128
MIN_EXP = -120


def nblk(n):
    return -(-n // BLK)


def plan(seq_len, n_new, table, free_pages, n_free, n_tok):
    """The page plan request by request; lists and numpy arrays, inputs unchanged."""
    B, max_blocks = table.shape
    table, free = table.copy(), list(free_pages[:n_free])
    tail = list(free_pages[n_free:])
    lens = list(seq_len)
    for b in range(B):
        if n_new[b] < 0:
            free += [int(table[b, j]) for j in range(nblk(lens[b]))]
            lens[b] = 0
    F = len(free)
    F0 = n_free
    pages_out = np.array((free + tail[F - F0:])[:len(free_pages)], dtype=np.int32)
    cu = np.zeros(B + 1, np.int64)
    start, out_len = np.zeros(B, np.int32), np.array(lens, dtype=np.int32)
    slot, req, pos = (np.full(n_tok, -1, np.int32) for _ in range(3))
    upto = taken = refused = 0
    for b in range(B):
        add = max(int(n_new[b]), 0)
        cu[b + 1] = cu[b] + add
        if n_new[b] < 0:
            continue
        old = lens[b]
        ok = old + add <= max_blocks * BLK and cu[b + 1] <= n_tok
        need = nblk(old + add) - nblk(old) if ok else 0
        upto += need
        ok = ok and (need == 0 or upto <= F)
        start[b] = old if ok else -1
        if not ok:
            refused += 1
            continue
        for j in range(nblk(old), nblk(old + add)):
            table[b, j] = free[F - 1 - taken]
            taken += 1
        for i in range(add):
            t, x = cu[b] + i, old + i
            slot[t], req[t], pos[t] = int(table[b, x // BLK]) * BLK + x % BLK, b, x
        out_len[b] = old + add
    return dict(table=table, free=pages_out, n_free=F - taken, cu=cu, start=start, len=out_len, slot=slot, req=req,
                pos=pos, refused=refused)


def e4m3_round(x):
    """Nearest e4m3 value (ties to even) of fp64 values within +-448; NaN stays."""
    a = np.maximum(np.abs(x), 2.0 ** -6)
    step = np.exp2(np.floor(np.log2(a)) - 3)
    return np.round(x / step) * step


def pow2_scale(amax):
    e = MIN_EXP
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(values, scale, k_new, v_new, slots, ktil=None, req=None, pos=None):
    """values [n_pages][H][2][64][128] (the e4m3 numbers), scale, ktil and rows as fp64 numpy;
    returns new copies.  Runs are found as the slots give them."""
    values, scale = values.copy(), scale.copy()
    ktil = None if ktil is None else ktil.copy()
    H = values.shape[1]
    t, T = 0, len(slots)
    while t < T:
        if slots[t] < 0 or slots[t] // BLK >= values.shape[0]:
            t += 1
            continue
        page, off = divmod(int(slots[t]), BLK)
        n = 1
        while t + n < T and off + n < BLK and slots[t + n] == slots[t] + n:
            n += 1
        for h in range(H):
            for kv, rows in enumerate((k_new, v_new)):
                x = rows[t:t + n, h]
                fin = np.isfinite(x)
                s = pow2_scale(np.abs(x[fin]).max() if fin.any() else 0.0)
                old = scale[page, h, kv]
                if off:
                    s = max(s, old)
                    values[page, h, kv, :off] = e4m3_round(values[page, h, kv, :off] * (old / s))
                with np.errstate(invalid="ignore"):
                    values[page, h, kv, off:off + n] = e4m3_round(np.where(fin, x, np.nan) / s)
                scale[page, h, kv] = s
            if ktil is not None:
                b, j = req[t], pos[t] // BLK
                if 0 <= b < ktil.shape[0] and 0 <= j < ktil.shape[2]:
                    ktil[b, h, j] = ((ktil[b, h, j] * off if off else 0.0) + k_new[t:t + n, h].sum(0)) / (off + n)
        t += n
    return values, scale, ktil


def attn(Q, values, scale, table, lens, blk_idx=None, count=None, sm_scale=None):
    """Q [B][Hq][128] fp64; returns O, lse and, for the tolerances, sum p |v| and the largest
    sum |q k| (scaled) of each row."""
    B, Hq, _ = Q.shape
    n_pages, H = values.shape[:2]
    G = Hq // H
    sm_scale = D ** -0.5 if sm_scale is None else sm_scale
    O, pv, lse, mag = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    for b in range(B):
        n = min(int(lens[b]), table.shape[1] * BLK)
        for g in range(H):
            blks = range(nblk(n)) if blk_idx is None else blk_idx[b, g, :max(0, min(int(count[b, g]), blk_idx.shape[2]))]
            K, V = [], []
            for j in blks:
                if not 0 <= j < table.shape[1] or j >= nblk(n) or not 0 <= table[b, j] < n_pages:
                    continue
                m = min(BLK, n - int(j) * BLK)
                page = table[b, j]
                K.append(values[page, g, 0, :m] * float(scale[page, g, 0]))
                V.append(values[page, g, 1, :m] * float(scale[page, g, 1]))
            if not K:
                continue
            K, V = np.concatenate(K), np.concatenate(V)
            for h in range(g * G, (g + 1) * G):
                s = sm_scale * (K @ Q[b, h])
                m = s.max()
                p = np.exp(s - m)
                lse[b, h] = m + np.log(p.sum())
                O[b, h] = p @ V / p.sum()
                pv[b, h] = p @ np.abs(V) / p.sum()
                mag[b, h] = (abs(sm_scale) * (np.abs(K) @ np.abs(Q[b, h]))).max()
    return O, lse, pv, mag


def assert_attn(O, lse, ref, n_max, what=""):
    """Against attn()'s answer.  A score is a sum of 128 products in fp32: off by at most
    128 * 2^-23 * sum |q k| in any order, even where sums are truncated; a weight is off by
    twice that and, rounded to 11 bits, 2^-11, and the exponential 2^-21; n_max weighted
    values are summed in fp32 (2^-23 each); the output is rounded to bf16 (2^-8 relative)."""
    Or, lr, pv, mag = ref
    O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
    e = 2.0 ** -16 * mag
    tol = (2 * e + 2.0 ** -11 + 2.0 ** -21 + n_max * 2.0 ** -23)[..., None] * pv + 2.0 ** -8 * np.abs(Or)
    off = np.abs(O - Or)
    assert np.isfinite(O).all(), what
    assert (off <= tol).all(), f"{what}: {off.max():.3e}, {(off - tol).max():.3e} over its bound"
    assert np.array_equal(np.isinf(lse), np.isinf(lr)), what
    fin = np.isfinite(lr)
    tol = e + n_max * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -21 * np.abs(np.where(fin, lr, 0))
    off = np.abs(lse[fin] - lr[fin])
    assert (off <= tol[fin]).all(), f"{what}: lse {off.max():.3e}"


def f8_values(pages: torch.Tensor) -> np.ndarray:
    return pages.detach().cpu().float().double().numpy()


def bf16(x, device):
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).to(device=device, dtype=torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()
