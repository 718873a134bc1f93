"""Frequencies of rotary positions, for ``binding.sparse_rope``."""
from __future__ import annotations

import math

import torch


def frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, scale: float = 1.0, original_len: int = 4096,
                slow_turns: float = 1.0, fast_turns: float = 32.0):
    """(inv_freq [rot_dim / 2] fp64, factor): pair i turns by inv_freq[i] = base^(-2 i / rot_dim) a position.

    ``scaling`` stretches the positions by ``scale`` for contexts longer than ``original_len``:
      "linear"  every frequency divided by scale;
      "base"    the base raised, base * scale^(rot_dim / (rot_dim - 2)): the slowest pair is divided by
                scale, the fastest stays;
      "parts"   pairs that turn fewer than slow_turns times in original_len positions divided by scale,
                those of more than fast_turns kept, a ramp in between, and the rotated values
                multiplied by factor = 0.1 ln(scale) + 1.
    """
    if rot_dim < 2 or rot_dim > 128 or rot_dim % 2:
        raise ValueError(f"rot_dim is even, from 2 to 128, got {rot_dim}")
    if not (base > 0 and math.isfinite(base) and scale > 0 and math.isfinite(scale)):
        raise ValueError("base and scale are finite and positive")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    if scaling == "base":
        if rot_dim == 2:
            raise ValueError("a single pair has no slower one to stretch")
        base = base * scale ** (rot_dim / (rot_dim - 2))
    f = base ** (-i / rot_dim)
    if scaling is None or scaling == "base":
        return f, 1.0
    if scaling == "linear":
        return f / scale, 1.0
    if scaling != "parts":
        raise ValueError(f"scaling is None, 'linear', 'base' or 'parts', got {scaling!r}")
    if not fast_turns > slow_turns:
        raise ValueError("fast_turns is above slow_turns")
    keep = ((original_len * f / (2 * math.pi) - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
    return f * keep + f / scale * (1 - keep), 0.1 * math.log(scale) + 1.0
