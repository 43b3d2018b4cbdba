"""Accuracy of the q/k norm where many bits count: far positions."""
from fractions import Fraction

import pytest
import torch

import plain_ops
from recurrent_state_quantization_lq_b200 import lq

pytestmark = pytest.mark.gpu
DEV = "cuda"
TWO_PI = 2 * Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)


def reduced(position, inv_freq):
    """position * inv_freq less whole turns, in exact arithmetic: radians within half a turn of 0."""
    turns = Fraction(position) * Fraction(inv_freq) / TWO_PI
    return float((turns - round(turns)) * TWO_PI)


@pytest.mark.parametrize("pairs,rot", [("neighbours", 128), ("half", 128), ("half", 120)])
@pytest.mark.parametrize("near", [1, 4096, 1000000, 2 ** 30, 2 ** 31 - 1, -2 ** 31])
def test_angles_keep_fp32_accuracy_at_any_position(pairs, rot, near):
    """Rows (1, 0) in every pair turn into (cos, sin) times one factor of the row, so atan2 of the result is the
    angle that was turned by.  Cosine and sine are within 2 ulp (at most 2 u absolute below 1) and take one rounding
    in the kernel's last turn and one in the output: 3 u each, across the circle at most 3 sqrt(2) u."""
    M, half = 40, rot // 2
    gen = torch.Generator().manual_seed(abs(near) % 1000)
    step = max(1, abs(near) // 2)
    pos = [min(2 ** 31 - 1, max(-2 ** 31, near - (1 if near > 0 else -1) * int(i))) for i in
           torch.randint(0, step, (M,), generator=gen).tolist()]
    freq = torch.rand(half, generator=gen, dtype=torch.float64) + 0.5          # near 1: no lost digits are hidden
    x = torch.zeros(M, 1, 128)
    first = torch.arange(half) * (1 if pairs == "half" else 2)
    second = first + half if pairs == "half" else first + 1
    x[..., first] = 1.0
    y, _ = lq.qk_norm_rotate(x.to(DEV), positions=torch.tensor(pos, dtype=torch.int32, device=DEV),
                             inv_freq=freq.to(DEV), pairs=pairs)
    y = y.double().cpu()[:, 0]
    want = torch.tensor([[reduced(p, f) for f in freq.tolist()] for p in pos], dtype=torch.float64)
    off = torch.atan2(y[:, second], y[:, first]) - want
    off = (off - 2 * torch.pi * torch.round(off / (2 * torch.pi))).abs()
    assert off.max() <= 3 * 2 ** 0.5 * plain_ops.U, float(off.max()) / plain_ops.U
