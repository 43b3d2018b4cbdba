"""The stateless operators on the paths that use them: a state that normalises
and rotates its q and k itself, and a layer pair (matrix state, then vector
state) over a prompt, decode tokens and a training step."""
import pytest
import torch

import plain_ops
from recurrent_state_quantization_lq_b200 import lq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def projections(T, B, H, d, gate, seed):
    """What a layer's projections give: rows of q, k and v together, log gates, input gates."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, B, 3, H, d, generator=gen).to(torch.bfloat16).to(DEV)
    g = -0.1 * torch.nn.functional.softplus(torch.randn(T, B, H, *([d] if gate == "channel" else []), generator=gen))
    beta = torch.sigmoid(torch.randn(T, B, H, generator=gen))
    return x, g.to(DEV), beta.to(DEV)


@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("rotate", [False, True])
def test_a_state_that_prepares_its_queries_and_keys(gate, rotate):
    """qk_norm= gives, bit for bit, what preparing q and k before each call gives."""
    T, P, B, H, d = 20, 13, 3, 4, 64
    x, g, beta = projections(T, B, H, d, gate, seed=1)
    how = {"norm": "l2", "q_scale": d ** -0.5}
    pos = None
    if rotate:
        how["inv_freq"] = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device=DEV) / (d // 2))
        pos = (torch.arange(T, dtype=torch.int32, device=DEV)[:, None] + 100 * torch.arange(B, dtype=torch.int32, device=DEV))
    at = lambda t: None if pos is None else pos[t].contiguous()  # noqa: E731
    q, k = lq.qk_norm_rotate(x[:, :, 0], x[:, :, 1], positions=pos, **how)
    v = x[:, :, 2].contiguous()
    outs = []
    for own in (False, True):
        st = lq.DecodeState(B, H, d, window=8, gate=gate, device=DEV, qk_norm=how if own else None)
        o = torch.empty(T, B, H, d, device=DEV)
        a, b = (x[:, :, 0], x[:, :, 1]) if own else (q, k)
        kw = (lambda t: {"positions": at(t)}) if own else (lambda t: {})
        st.prefill_tokens(a[:P], b[:P], v[:P], g[:P], beta[:P], out=o[:P], **kw(slice(0, P)))
        for t in range(P, T):
            st.decode_step(a[t], b[t], v[t], g[t], beta[t], out=o[t], **kw(t))
            if st.fill == 8:
                st.flush()
        assert st.device_status() == lq.LQ_OK
        outs.append(o)
    assert torch.equal(*outs)
    assert torch.isfinite(outs[0]).all() and outs[0].abs().max() > 0


def test_positions_want_a_norm():
    st = lq.DecodeState(1, 2, 64, device=DEV)
    st.prefill(None)
    x, g, beta = projections(1, 1, 2, 64, "scalar", seed=2)
    a = x[0, :, 0].contiguous()
    with pytest.raises(AssertionError, match="positions"):
        st.decode_step(a, a, a, g[0], beta[0], positions=torch.zeros(1, dtype=torch.int32, device=DEV))


def test_two_layers_over_a_prompt_and_decode_tokens():
    """A ragged batch: prompts of different lengths through the matrix-state layer (q, k prepared by the
    state) and, on its outputs, the vector-state layer; then decode tokens of the active sequences.
    Splitting the prompt differently changes nothing but rounding in the second layer."""
    T, B, H, d, steps = 40, 4, 2, 64, 5
    x, g, beta = projections(T + steps, B, H, d, "scalar", seed=3)
    lengths = torch.tensor([40, 7, 0, 23], dtype=torch.int32, device=DEV)
    v = x[:, :, 2].contiguous()
    st = lq.DecodeState(B, H, d, window=8, ragged=True, device=DEV, qk_norm={})
    st.prefill(None)
    o = torch.zeros(T, B, H, d, device=DEV)
    st.prefill_sequences_tokens(x[:T, :, 0], x[:T, :, 1], v[:T], g[:T], beta[:T],
                                torch.ones(B, dtype=torch.uint8, device=DEV), lengths=lengths, out=o)
    y, h = lq.gated_scan(o, g[:T], beta[:T], lengths=lengths)
    want = plain_ops.scan(o, g[:T], beta[:T], None, lengths)
    plain_ops.check(y, want["out"], torch.float32, "prompt")
    plain_ops.check(h, want["h_last"], torch.float32, "state")
    active = torch.tensor([1, 0, 1, 1], dtype=torch.uint8, device=DEV)
    one = active.to(torch.int32)                              # a decode token is a length of one, or none
    for t in range(T, T + steps):
        before = h.clone()
        ot = torch.zeros(B, H, d, device=DEV)
        st.decode_step(x[t, :, 0], x[t, :, 1], v[t], g[t], beta[t], out=ot, active=active)
        st.flush()
        y, h = lq.gated_scan(ot[None], g[t:t + 1], beta[t:t + 1], h, lengths=one, h_last=h)
        want = plain_ops.scan(ot[None], g[t:t + 1], beta[t:t + 1], before, one)
        plain_ops.check(y, want["out"], torch.float32, f"token {t}")
        plain_ops.check(h, want["h_last"], torch.float32, f"state after {t}")
        assert torch.equal(h[1], before[1]) and (y[0, 1] == 0).all()
    assert st.device_status() == lq.LQ_OK


def test_a_training_step_through_both_operators():
    """Gradients through scan(v = normed k) back to the projection, against the 64-bit chain of formulas."""
    T, B, H, d = 70, 2, 2, 64
    x, g, beta = projections(T, B, H, d, "scalar", seed=4)
    x = x.float()
    w = 1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(5)).to(DEV)
    how = {"norm": "rms", "weight_k": w, "weight_q": w}
    q, k = x[:, :, 0], x[:, :, 1]
    qn, kn = lq.qk_norm_rotate(q, k, **how)
    marks = lq.gated_scan_checkpoints(kn, g)
    y, _ = lq.gated_scan(kn, g, beta, checkpoints=marks)
    dy = qn                                                    # the loss sum(y q) with q's part held
    gkn, gg, gb, _ = lq.gated_scan_backward(dy, kn, g, beta, checkpoints=marks)
    _, gk, _, gw = lq.qk_norm_rotate_backward(torch.zeros_like(qn), gkn, q, k, **how)

    kd, gd, bd, wd = (t.double().cpu().requires_grad_() for t in (k, g, beta, w))
    n = kd / torch.sqrt(kd.square().mean(-1, keepdim=True) + 1e-6) * wd
    h, loss = torch.zeros(B, H, d, dtype=torch.float64), 0.0
    for t in range(T):
        h = gd[t].exp()[..., None] * h + bd[t][..., None] * n[t]
        loss = loss + (h * qn[t].double().cpu()).sum()
    loss.backward()
    for got, want in ((gk, kd.grad), (gg, gd.grad), (gb, bd.grad), (gw, wd.grad)):
        # two operators' roundings: each is below 200 u of the largest value here (70 tokens, 64 channels)
        assert (got.double().cpu() - want).abs().max() <= 400 * plain_ops.U * want.abs().max()
