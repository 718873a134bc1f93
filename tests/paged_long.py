"""The paged attention over long lists: a plain implementation in 64 bits, and a bound of the
kernel's answer that a lost or repeated tile of 64 tokens among 131 072 does not meet."""
from __future__ import annotations

import numpy as np

BLK, D = 64, 128


def tokens(values, scale, table, n, head):
    """Keys and values [n][128] of one request's head, fp64."""
    pages = table[:-(-n // BLK)]
    K, V = (values[pages, head, kv] * scale[pages, head, kv][:, None, None] for kv in (0, 1))
    return K.reshape(-1, D)[:n], V.reshape(-1, D)[:n]


def attend(Q, K, V, sm_scale=D ** -0.5, times=None):
    """Q [G][128] over tokens, each counted `times` (once): O, lse and, for the bound, the root of the
    sum of (p v)^2, and the largest sum |q k| (scaled)."""
    s = sm_scale * (Q @ K.T)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m) * (1 if times is None else times)
    l = p.sum(1, keepdims=True)
    spread = np.sqrt((p / l) ** 2 @ V ** 2)
    mag = abs(sm_scale) * (np.abs(Q) @ np.abs(K).T).max(1)
    return p @ V / l, (m + np.log(l))[:, 0], spread, mag


def assert_close(O, lse, ref, what=""):
    """For values whose signs are independent of keys and queries (random ones).  A weight is off by
    at most w: twice its score's error e (a sum of 128 products in fp32: 128 * 2^-23 * sum |q k|), the
    exponential's 2^-21, 2^-11 from rounding to f16, and 512 additions in fp32 at most between it
    and the output (a warp's tiles, four steps each, the warps, two merges of 32 states):
    2^-14.  The signs make a sum of such errors a random walk: 8 standard deviations, which one
    element in 10^13 passes.  The sum of the weights is off by e, 2^-21 and 2^-14, and the
    output is rounded to bf16 (2^-8)."""
    Or, lr, spread, mag = ref
    e = 2.0 ** -16 * mag
    w, sums = 2 * e + 2.0 ** -21 + 2.0 ** -11 + 2.0 ** -14, e + 2.0 ** -21 + 2.0 ** -14
    tol = 8 * w[:, None] * spread + (2.0 ** -8 + sums[:, None]) * np.abs(Or)
    off = np.abs(np.asarray(O, dtype=np.float64) - Or)
    assert (off <= tol).all(), f"{what}: {(off / tol).max():.2f} of its bound"
    off, tol = np.abs(np.asarray(lse, dtype=np.float64) - lr), sums + 2.0 ** -21 * np.abs(lr)
    assert (off <= tol).all(), f"{what}: lse {(off / tol).max():.2f} of its bound"
