"""The angle of a far position, seen where the sine is next to zero: there a result's size is that of the angle."""
from decimal import Decimal, getcontext

import pytest
import torch

from block_sparse_long_pool_gb300 import binding

pytestmark = pytest.mark.gpu
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def small_angles(f, n, count=200000):
    """Positions next to 2^31 whose angle is closest to whole turns, and the angles in turns, from integers of 2^-128."""
    getcontext().prec = 110
    unit = 1 << 128
    F = int((Decimal(f) / (2 * PI) * unit).to_integral_value())
    found = []
    for pos in range(2 ** 31 - count, 2 ** 31):
        at = (pos * F + unit // 2) % unit - unit // 2
        found.append((abs(at), pos, at / unit))
    return [(pos, x) for _, pos, x in sorted(found)[:n]]


@pytest.mark.parametrize("f", [1.0, -1.0, 0.1, -0.1, -0.75, 0.75, -1e-4, -0.37, -2.5, 100.0, -100.0, 1234567.0, -1234567.0])
def test_angles_near_whole_turns(f):
    found = small_angles(f, 12)
    n = len(found)
    pos = torch.tensor([p for p, _ in found], dtype=torch.int64, device="cuda").to(torch.int32)
    x = torch.tensor([t for _, t in found], dtype=torch.float64, device="cuda") * (2 * torch.pi)
    assert x.abs().max() < 1e-3
    Q = torch.zeros((n, 1, 128), dtype=torch.bfloat16, device="cuda")
    Q[..., 1] = 1.0   # a = 0, b = 1: -sin x, cos x
    out = torch.empty_like(Q)
    binding.sparse_rope(Q, None, pos, torch.tensor([f], dtype=torch.float64, device="cuda"), out, None)
    want = -torch.sin(x)
    # the frequency in turns is off by 1.1 units of 2^-64, so an angle by 1.1 * 2^31 of them; the upper 32 bits are
    # taken of it (2^-32 turns); sincospi is off by two units in the last place; bf16's half step
    tol = want.abs() * (2.0 ** -8 + 2.0 ** -21) + 2 * torch.pi * (1.1 * 2.0 ** -33 + 2.0 ** -32)
    err = (out[:, 0, 0].double() - want).abs()
    assert (err <= tol).all(), f"{(err / tol).max().item():.3g} bounds, angles off by {(err / 6.2832).max().item():.3g} turns"
    assert ((out[:, 0, 1].double() - torch.cos(x)).abs() <= 2.0 ** -8).all()
