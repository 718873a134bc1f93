"""Chunk attention's weights and row sums where scores and value scales are far apart."""
import pytest
import torch

from block_sparse_long_pool_gb300 import binding
from tests.chunk_utils import BLK, D, Chunk

pytestmark = pytest.mark.gpu


def ws(c):
    return binding.paged_chunk_workspace(c.B, c.H_q, c.H_kv)


@pytest.mark.parametrize("above", [11.5, 14.5])
@pytest.mark.parametrize("at", [0, 70])
def test_small_weights_behind_a_token_of_none(at, above):
    # a token `above` nats over all others whose values are next to nothing: the others' weights carry the output.
    # More items than a GPU has SMs, so that most of them are one CTA's
    B, H, G = 40, 4, 2
    c = Chunk([2000] * B, [3] * B, H, G, seed=31)
    c.scale.fill_(1.0)
    c.pages.copy_(c.pages.float().abs().to(torch.float8_e4m3fn))   # positive values: rounding of the weights does not average out
    c.Q.zero_()
    c.Q[..., 0] = 1.0
    c.pages[:, :, 0] = 0.0
    c.pages[:, :, 0, :, 0] = -0.5
    for b in range(B):
        p = int(c.table[b, at // BLK])
        c.pages[p, :, 0, at % BLK, 0] = above - 0.5
        c.pages[p, :, 1, at % BLK] = 2.0 ** -9
    for b in range(B):   # (any bytes behind the last token)
        c.pages[int(c.table[b, 2003 // BLK]), :, :, 2003 % BLK:] = float("nan")
    c.call(ws(c), scale=1.0)
    torch.cuda.synchronize()
    assert c.status.item() == 0
    O, _, _, _ = c.expected(1.0)
    # Weights in f16 relative to 2^-8 of the largest of a page: 2^-11 of each where that is 2^-14 or more, so down to 2^-22 of
    # the largest (14.5 nats are 2^20.9), and 2^-33 of the largest below.  Scores are exact but for the product with log2 e and
    # the exponent's sum (2^-23 of 21 each, times ln 2), 2^x by 2^-22: 2^-17 together.  Values positive: a relative bound.
    # O in bf16: 2^-8.
    tol = O.abs() * (2.0 ** -8 + (2.0 ** -11 + 2.0 ** -16) * (1 + 2.0 ** -8))
    tol = tol + 2.0 ** -33 * 448 * 2003
    err = (c.O.double() - O).abs()
    assert (err <= tol).all(), f"O off by {(err / O.abs()).max().item():.3g}"


@pytest.mark.parametrize("high", [88.0, 200.0])
@pytest.mark.parametrize("vs", [2.0 ** -120, 0.0])
@pytest.mark.parametrize("last", ["high", "low"])
def test_a_page_of_small_values_far_above(high, vs, last):
    # scores 2^127 and more above the first page's, with values that add next to nothing; then a page that does
    # (where it is as high), or one that is far below again
    c = Chunk([170], [20], 1, 4, seed=32)
    c.scale.fill_(1.0)
    c.Q.zero_()
    c.Q[..., 0] = 1.0
    c.pages[:, :, 0] = 0.0
    c.pages[int(c.table[0, 1]), :, 0, :, 0] = high
    if last == "high":
        c.pages[int(c.table[0, 2]), :, 0, :, 0] = high
    c.pages[int(c.table[0, 2]), :, :, 62:] = float("nan")
    c.scale[int(c.table[0, 1]), :, 1] = vs
    c.call(ws(c), scale=1.0)
    c.check(1.0)
    assert c.lse.isfinite().all() and (c.lse > torch.tensor(high).to(torch.float8_e4m3fn).item()).all()


@pytest.mark.parametrize("start,new", [([170], [20]), ([9000], [3]), ([150] * 90, [2] * 90)])
@pytest.mark.parametrize("exp", [18, 21, 24, 27, 28, 30, 40, 90, 110])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("vs", [-6, 30])
def test_scores_of_any_size(start, new, exp, sign, vs):
    # scores of 2^exp and 9/8 of it, of either sign: the tokens with the largest share the row, all others are nothing.  Their
    # number is two or three, in one page and in others, whose value scales differ
    c = Chunk(start, new, 2, 4, seed=33)
    n = start[0]
    few = [3, 5, 100]
    c.Q.zero_()
    c.Q[..., 0] = 1.0
    c.pages[:, :, 0] = 0.0
    c.pages[:, :, 0, :, 0] = 8.0 if sign > 0 else -9.0
    c.scale[..., 0] = 2.0 ** (exp - 3)
    c.scale[..., 1] = 2.0 ** vs
    want = torch.zeros((c.B, 2, D), dtype=torch.float64, device="cuda")
    for b in range(c.B):
        c.scale[int(c.table[b, 1]), :, 1] = 2.0 ** (vs - 3)
        for t in few:
            p = int(c.table[b, t // BLK])
            c.pages[p, :, 0, t % BLK, 0] = 9.0 if sign > 0 else -8.0
            want[b] += c.pages[p, :, 1, t % BLK].double() * c.scale[p, :, 1].double()[:, None] / len(few)
        end = start[b] + new[b]
        c.pages[int(c.table[b, end // BLK]), :, :, end % BLK:] = float("nan")   # (any bytes behind the last token)
    c.call(ws(c), scale=1.0)
    torch.cuda.synchronize()
    assert c.status.item() == 0
    top = (9.0 if sign > 0 else -8.0) * 2.0 ** (exp - 3)
    row = 0
    for b in range(c.B):
        r = slice(row, row + new[b])
        row += new[b]
        w = want[b].repeat_interleave(4, 0)
        # the largest scores have the same bits, so their weights are alike but for 2^x (2^-22) and f16 (2^-11), where a
        # reference in fp32 leaves 2^0 to 2^-8 of them; the others' are below 2^(-2^14).  O in bf16: 2^-8
        size = w.abs() + 448 * 2.0 ** vs
        assert ((c.O[r].double() - w).abs() <= w.abs() * 2.0 ** -8 + size * (2.0 ** -11 + 2.0 ** -18) * (1 + 2.0 ** -8)).all()
        # lse: base 2 and back, three roundings of the largest score, and ln 3
        lse = top + torch.tensor(float(len(few)), dtype=torch.float64).log().item()
        assert ((c.lse[r].double() - lse).abs() <= abs(lse) * 2.0 ** -21 + 2.0 ** -16).all()
