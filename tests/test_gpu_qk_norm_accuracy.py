"""Accuracy of the q/k norm where many bits count: far positions, and weight
gradients over more tokens than the backward kernel takes in one round."""
from fractions import Fraction

import pytest
import torch

import plain_ops
from recurrent_state_quantization_lq_b200 import lq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
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


def test_weight_gradients_round_once_over_the_tokens():
    """Rows of ones are their own norm, so dw = sum over the rows of dy.  With gradients of 18 bits a CTA's part (8 row
    groups of one or two rows) is exact in FP32; the sum over the CTAs is not, and must be rounded once."""
    M, d = 9000, 256
    gen = torch.Generator().manual_seed(1)
    x = torch.ones(M, 1, d, device=DEV)
    dy = ((2 ** 17 + torch.randint(0, 2 ** 17, (M, 1, d), generator=gen)).double() / 2 ** 17).to(F32).to(DEV)
    w = torch.ones(d, device=DEV)
    how = {"norm": "rms", "eps": 1e-30, "weight_q": w, "weight_k": w}
    for y in lq.qk_norm_rotate(x, x, **how):
        assert (y == 1).all()
    _, _, gwq, gwk = lq.qk_norm_rotate_backward(dy, dy, x, x, **how)
    want = dy.double().sum((0, 1)).to(F32)
    assert torch.equal(gwq, want) and torch.equal(gwk, want)


@pytest.mark.parametrize("heads,rounds", [(1, 64), (4, 16), (48, 2)])
def test_weight_gradients_do_not_lose_more_with_the_rounds(heads, rounds):
    """Rows of ones and one gradient everywhere: dw = M heads g.  A thread takes heads x rounds rows, and for this g
    plain FP32 additions round with one sign, up to 0.5 u of each partial sum: n of them leave up to
    sum_i 0.5 u i / n = 0.25 (n + 1) u, the same in every thread.  Allowed: that of 32 rows, or of one token's heads,
    that of the CTA's 8 rows of threads, and the roundings of both sums and of the result, 1.5 u."""
    M, d, g = rounds * 8192, 256, float.fromhex("0x1.f08ccp+0")
    x, dy, w = torch.ones(M, heads, d, device=DEV), torch.full((M, heads, d), g, device=DEV), torch.ones(d, device=DEV)
    gw = lq.qk_norm_rotate_backward(dy, None, x, norm="rms", eps=1e-30, weight_q=w)[2]
    off = (gw.double().cpu() / (M * heads * g) - 1).abs().max()
    assert off <= (0.25 * (max(32, heads) + 1 + 8 + 1) + 1.5) * plain_ops.U, float(off) / plain_ops.U


@pytest.mark.parametrize("M,hq,hk,d,rot,pairs", [(8192 + 5, 1, 1, 256, 256, "half"), (16384 + 3, 1, 2, 128, 128, "half"),
                                                 (16384 + 3, 2, 1, 128, 64, "neighbours"), (32768 + 9, 1, 1, 64, 36, "half"),
                                                 (2 * 16384 + 1, 1, 0, 100, 24, "half"), (2 * 32768 + 77, 2, 1, 50, 0, "half")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_tokens_than_one_round_of_the_backward_kernel(M, hq, hk, d, rot, pairs, dtype):
    """The grid is capped at 1024 CTAs (1024 x 8, 16 or 32 rows): threads carry their weight gradients over rounds,
    the last of which is partly dead.  dw is held to the additions that are made: a thread's rows, one by one, and
    32 more of the CTA's, and three roundings of larger sums: (48 + at most 41) u of the sum of absolute values, 5.3e-6.  One row's part is
    1 / (M heads) of that sum, 7.6e-6 and more."""
    gen = torch.Generator().manual_seed(M)
    on = lambda *s: torch.randn(*s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    q, gq = on(M, hq, d), on(M, hq, d)
    k, gk = (on(M, hk, d), on(M, hk, d)) if hk else (None, None)
    how = {"norm": "rms", "pairs": pairs, "q_scale": 0.5, "weight_q": torch.randn(d, generator=gen).to(DEV)}
    if hk:
        how["weight_k"] = torch.randn(d, generator=gen).to(DEV)
    if rot:
        how["positions"] = torch.randint(0, 5000, (M,), generator=gen, dtype=torch.int32).to(DEV)
        how["inv_freq"] = (10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)).to(DEV)
    got = lq.qk_norm_rotate_backward(gq, gk, q, k, **how)
    lanes = 1
    while 8 * lanes < d:
        lanes *= 2
    rounds = -(-M // (1024 * (256 // lanes)))
    assert rounds > 1
    for i, (x, dy, heads, scale) in enumerate(((q, gq, hq, 0.5), (k, gk, hk, 1.0))):
        if x is None:
            continue
        want = plain_ops.qk(x, how.get("positions"), how.get("inv_freq"), how["weight_" + "qk"[i]], "rms", 1e-6, pairs,
                            scale, dy)
        assert torch.isfinite(got[i]).all() and torch.isfinite(got[2 + i]).all()
        plain_ops.check(got[i], want["dx"], dtype, "dx")
        value, loose = want["dw"]
        C = 2 * plain_ops.C_QK
        plain_ops.check(got[2 + i], (value, loose * (C + rounds * heads + 32 + 3) / (C + M * heads)), F32, "dw")
