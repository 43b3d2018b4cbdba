"""The q/k norm with rotation and its gradients against their 64-bit formulas."""
import pytest
import torch

import plain_ops
from recurrent_state_quantization_lq_b200 import inputs, lq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def case(M, hq, hk, d, rot=0, dtype=BF, weights=True, far=5000, seed=0):
    gen = torch.Generator().manual_seed(seed)
    on = lambda x: x.to(DEV)  # noqa: E731
    c = {"q": on(torch.randn(M, hq, d, generator=gen).to(dtype)), "k": on(torch.randn(M, hk, d, generator=gen).to(dtype)),
         "gq": on(torch.randn(M, hq, d, generator=gen).to(dtype)), "gk": on(torch.randn(M, hk, d, generator=gen).to(dtype))}
    how = {"q_scale": 0.25}
    if weights:
        how["weight_q"], how["weight_k"] = on(torch.randn(d, generator=gen)), on(torch.randn(d, generator=gen))
    if rot:
        how["positions"] = on(torch.randint(0, far, (M,), generator=gen, dtype=torch.int32))
        how["inv_freq"] = on(10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot))
    return c, how


def verify(c, how, backward=True):
    q, k = lq.qk_norm_rotate(c["q"], c["k"], **how)
    g = lq.qk_norm_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], **how) if backward else None
    for i, (x, y, dy, w, scale) in enumerate(((c["q"], q, c["gq"], how.get("weight_q"), how["q_scale"]),
                                              (c["k"], k, c["gk"], how.get("weight_k"), 1.0))):
        want = plain_ops.qk(x, how.get("positions"), how.get("inv_freq"), w, how.get("norm", "l2"),
                            how.get("eps", 1e-6), how.get("pairs", "half"), scale, dy)
        plain_ops.check(y, want["y"], y.dtype, "qk"[i])
        if backward:
            plain_ops.check(g[i], want["dx"], x.dtype, "gradient of " + "qk"[i])
            assert (g[2 + i] is None) == (w is None)
            if w is not None:
                plain_ops.check(g[2 + i], want["dw"], F32, "weight gradient of " + "qk"[i])
    return (q, k), g


@pytest.mark.parametrize("d", [1, 2, 3, 8, 10, 16, 24, 32, 40, 63, 64, 72, 80, 96, 100, 128, 192, 250, 256])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_head_sizes(d, norm):
    c, how = case(37, 3, 2, d, rot=d // 2 * 2, dtype=F32 if d % 3 == 0 else BF, seed=d)
    verify(c, {**how, "norm": norm})


@pytest.mark.parametrize("pairs", ["half", "neighbours"])
@pytest.mark.parametrize("rot", [0, 2, 6, 16, 32, 40, 64, 96, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_partial_rotations(pairs, rot, dtype):
    c, how = case(50, 4, 2, 128, rot=rot, dtype=dtype, seed=rot)
    verify(c, {**how, "pairs": pairs, "norm": "rms"})


@pytest.mark.parametrize("M,hq,hk", [(1, 1, 1), (1, 32, 8), (2, 5, 5), (7, 3, 1), (8, 64, 4), (65, 1, 3), (300, 8, 8), (3000, 2, 1)])
@pytest.mark.parametrize("weights", [False, True])
def test_tokens_and_heads(M, hq, hk, weights):
    c, how = case(M, hq, hk, 64, rot=64, weights=weights, seed=M)
    verify(c, how)


def test_far_and_negative_positions():
    c, how = case(6, 2, 2, 64, rot=64, dtype=F32, seed=3)
    how["positions"] = torch.tensor([0, 1, -1, 1000000, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    verify(c, how)


def test_rows_of_zeros_and_of_extremes():
    c, how = case(5, 2, 2, 64, rot=32, dtype=F32, weights=False, seed=4)
    c["q"][0] = 0.0
    c["q"][1] = 1e-30                                 # squares underflow: eps decides
    c["q"][2, 0] = 1e15
    c["q"][3, 1, 7] = float("nan")
    q, k = lq.qk_norm_rotate(c["q"], c["k"], **how)
    assert (q[0] == 0).all() and torch.isfinite(q[:3]).all() and torch.isfinite(q[3, 0]).all()
    assert torch.isnan(q[3, 1]).all() and torch.isfinite(k).all() and torch.isfinite(q[4]).all()
    verify({n: x[[0, 1, 2, 4]] for n, x in c.items()},
           {**how, "positions": how["positions"][[0, 1, 2, 4]]})


def test_views_of_a_fused_projection():
    """Aligned and unaligned views give what packed copies give; outputs may be views too."""
    M, hq, hk, d = 40, 4, 2, 64
    c, how = case(M, hq, hk, d, rot=48, seed=5)
    want, grads = verify(c, how)
    for extra in (0, 8, 3):
        x = torch.zeros(M, (hq + 2 * hk) * d + extra, dtype=BF, device=DEV)
        q, k = x[:, extra:extra + hq * d].unflatten(1, (hq, d)), x[:, extra + hq * d:extra + (hq + hk) * d].unflatten(1, (hk, d))
        q.copy_(c["q"])
        k.copy_(c["k"])
        got = lq.qk_norm_rotate(q, k, **how)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), extra
        back = lq.qk_norm_rotate_backward(c["gq"], c["gk"], q, k, **how)
        for a, w in zip(back[:2], grads[:2]):
            assert torch.equal(a, w), extra
        into = lq.qk_norm_rotate(q, k, q_out=q, k_out=k, **how)           # in place
        assert into[0] is q and all(torch.equal(a, b) for a, b in zip(into, want)), extra
        assert (x[:, extra + (hq + hk) * d:] == 0).all() and (x[:, :extra] == 0).all()


def test_queries_alone_and_leading_dimensions():
    T, B, H, d = 5, 3, 4, 64
    c, how = case(T * B, H, 1, d, rot=d, weights=False, seed=6)
    q4, pos = c["q"].view(T, B, H, d), how["positions"].view(T, B)
    want = lq.qk_norm_rotate(c["q"], c["k"], **how)[0]
    got, none = lq.qk_norm_rotate(q4, **{**how, "positions": pos})
    assert none is None and torch.equal(got.view(-1, H, d), want)
    gq, none, _, _ = lq.qk_norm_rotate_backward(c["gq"].view(T, B, H, d), None, q4, **{**how, "positions": pos})
    assert none is None and gq.shape == q4.shape
    with pytest.raises(AssertionError):       # the tokens of a transposed view are not one run
        lq.qk_norm_rotate(q4.transpose(0, 1), **{**how, "positions": pos.t().contiguous()})


def test_a_key_weight_without_keys():
    c, how = case(20, 3, 1, 64, seed=12)
    want = lq.qk_norm_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], **how)
    gq, none, gwq, gwk = lq.qk_norm_rotate_backward(c["gq"], None, c["q"], **how)
    assert none is None and gwk is None and torch.equal(gq, want[0]) and torch.equal(gwq, want[2])


def test_in_place_backward():
    c, how = case(30, 3, 2, 128, rot=128, seed=7)
    want = lq.qk_norm_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], **how)
    got = lq.qk_norm_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], grad_q=c["gq"], grad_k=c["gk"], **how)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_no_tokens():
    c, how = case(0, 2, 2, 64, rot=64)
    q, k = lq.qk_norm_rotate(c["q"], c["k"], **how)
    assert q.shape == (0, 2, 64) and k.shape == (0, 2, 64)
    _, _, gwq, gwk = lq.qk_norm_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], **how)
    assert (gwq == 0).all() and (gwk == 0).all()


def test_gradients_follow_differences():
    c, how = case(9, 2, 1, 32, rot=16, dtype=F32, seed=8)
    grads = lq.qk_norm_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], **how)

    def loss(x, w, scale, dy):
        y = plain_ops.qk(x, how["positions"], how["inv_freq"], w, "l2", 1e-6, "half", scale)["y"][0]
        return float((y * dy.double().cpu()).sum())

    e = 1e-5
    for x, w, s, dy, gx, gw in ((c["q"], how["weight_q"], 0.25, c["gq"], grads[0], grads[2]),
                                (c["k"], how["weight_k"], 1.0, c["gk"], grads[1], grads[3])):
        gen = torch.Generator().manual_seed(1)
        x, w = x.double().cpu(), w.double().cpu()
        vx, vw = (torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in (x, w))
        want = plain_ops.qk(x, how["positions"], how["inv_freq"], w, "l2", 1e-6, "half", s, dy)
        for diff, got, way, ref in (((loss(x + e * vx, w, s, dy) - loss(x - e * vx, w, s, dy)) / (2 * e), gx, vx, want["dx"]),
                                    ((loss(x, w + e * vw, s, dy) - loss(x, w - e * vw, s, dy)) / (2 * e), gw, vw, want["dw"])):
            slope = float((got.double().cpu() * way).sum())
            lim = float((ref[1] * way.abs()).sum()) + 1e-6 * float((ref[0] * way).abs().sum())
            assert abs(diff - slope) <= lim, (diff, slope, lim)


def test_other_streams_and_graphs():
    c, how = case(64, 4, 2, 128, rot=128, seed=9)
    want = [*lq.qk_norm_rotate(c["q"], c["k"], **how),
            *lq.qk_norm_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], **how)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [*lq.qk_norm_rotate(c["q"], c["k"], stream=s, **how),
           *lq.qk_norm_rotate_backward(c["gq"], c["gk"], c["q"], c["k"], stream=s, **how)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    static = {n: torch.zeros_like(x) for n, x in c.items()}
    static["q"].fill_(1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = [*lq.qk_norm_rotate(static["q"], static["k"], **how),
               *lq.qk_norm_rotate_backward(static["gq"], static["gk"], static["q"], static["k"], **how)]
    for n, x in c.items():
        static[n].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_it_makes_the_inputs_of_the_seeded_workloads():
    """L2 norm without rotation is the recipe that the decode workloads' q and k come from."""
    gen = torch.Generator().manual_seed(1)
    raw = torch.randn(6, 4, 8, 128, generator=gen)
    q, _ = lq.qk_norm_rotate(raw.to(DEV), norm="l2", eps=1e-12)
    want = raw.double() / raw.double().norm(dim=-1, keepdim=True)
    plain_ops.check(q, (want, plain_ops.C_QK * plain_ops.U * want.abs()), F32)
    assert inputs.WORKLOADS["gdn_b64_h32_d128_w64"].d_k == 128
