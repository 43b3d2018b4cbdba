"""Growing states: the gated scan over the stated range of gates, a sum of 80 over consecutive tokens."""
import pytest
import torch

import plain_ops
from recurrent_state_quantization_lq_b200 import lq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,B,H", [(20, 1, 2), (400, 1, 2), (400, 40, 16), (3000, 1, 3)])
@pytest.mark.parametrize("chan", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gates_that_grow_over_a_state_of_zeros(T, B, H, chan, dtype):
    """Padding on the left (no tokens, a zero state, open gates) and then growth, up to the stated sum."""
    d = 64
    gen = torch.Generator().manual_seed(T + B)
    v, dy = (torch.randn(T, B, H, d, generator=gen) for _ in range(2))
    v[:T // 2] = 0.0
    v, dy = v.to(dtype).to(DEV), dy.to(dtype).to(DEV)
    # a sum of at most 79.9 over all tokens (rounded sums of T values near it stay below 80)
    g = torch.rand(T, B, H, *([d] if chan else []), generator=gen)
    g = (79.9 * g / g.sum(0)).to(DEV)
    beta = torch.rand(T, B, H, generator=gen).to(DEV)
    dh = torch.zeros(B, H, d, device=DEV)
    dy[:T // 2] = 0.0                 # keeps gradients times states inside FP32
    marks = lq.gated_scan_checkpoints(v, g)
    out, last = lq.gated_scan(v, g, beta, checkpoints=marks)
    got = {"out": out, "h_last": last}
    got |= dict(zip(("grad_v", "grad_g", "grad_beta", "grad_h0"),
                    lq.gated_scan_backward(dy, v, g, beta, checkpoints=marks, grad_last=dh)))
    want = plain_ops.scan(v, g, beta, None, None, dy, dh)
    assert (out[:T // 2] == 0).all()
    for n, w in want.items():
        assert torch.isfinite(got[n]).all(), n
        plain_ops.check(got[n], w, got[n].dtype, n)


def test_an_infinite_state_stays_in_its_channel():
    """Whatever the split makes of it (an infinity, or NaN where a run's gates underflow), it is not finite again."""
    T, B, H, d = 2000, 1, 2, 64
    gen = torch.Generator().manual_seed(5)
    v = torch.randn(T, B, H, d, generator=gen).to(DEV)
    g = -torch.rand(T, B, H, generator=gen).to(DEV)
    h0 = torch.zeros(B, H, d, device=DEV)
    h0[0, 0, 3] = float("inf")
    v[777, 0, 1, 9] = float("-inf")
    out, last = lq.gated_scan(v, g, None, h0)
    assert not torch.isfinite(out[:, 0, 0, 3]).any() and not torch.isfinite(out[777:, 0, 1, 9]).any()
    assert torch.isfinite(out[:777, 0, 1]).all()
    rest = torch.ones(H, d, dtype=torch.bool, device=DEV)
    rest[0, 3] = rest[1, 9] = False
    assert torch.isfinite(out[:, 0][:, rest]).all() and torch.isfinite(last[0][rest]).all()
