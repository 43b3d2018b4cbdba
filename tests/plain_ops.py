"""Plain 64-bit forms of the stateless operators, with bounds on FP32 rounding.

Each reference returns, beside every result, a bound on the error that FP32
arithmetic may leave in it.  u = 2^-24 is FP32's unit roundoff.

Scan.  With S_t = a_t S_{t-1} + |x_t| (the recurrence of absolute values), one
token's work (exp within 2 ulp = 4 u, the products and sums of the recurrence,
and the few products that compose the maps of token runs) leaves at most
C u S_t, C = 16, and later gates carry it on: the total is at most C u R_t with
R_t = a_t R_{t-1} + S_t.  The backward recurrence has the same form.  A product
of two such values has the products of each bound with the other's absolute
value, and a sum over d channels adds one u per term and level (at most 16).

q/k norm.  r = (sum x^2 + eps)^(-1/2): at most 13 roundings in the sum, halved
by the root, 2 ulp of rsqrt: within 12 u.  cos and sin are within 4 u absolute
(2 ulp, and an angle rounded at pi 2^-24).  A rotated pair is thus within
C u (|u_a| + |u_b|), C = 24, and so on through the products.
"""
import torch

U = 2.0 ** -24
C_SCAN = 16
C_QK = 24


def step(dtype) -> float:
    """Half a step of the type, relative."""
    return torch.finfo(dtype).eps / 2


def run_recurrence(a, x, h):
    """h_t = a_t h_{t-1} + x_t over the first axis; every h_t."""
    out = torch.empty(torch.broadcast_shapes(a.shape, x.shape), dtype=x.dtype)
    for t in range(x.shape[0]):
        h = a[t] * h + x[t]
        out[t] = h
    return out


def scan(v, g, beta, h0, lengths, grad_out=None, grad_last=None):
    """{name: (value, bound)} in FP64 on the CPU, in the layouts of the calls; tokens past a length are zero."""
    T, B, H, d = v.shape
    v, g = v.double().cpu(), g.double().cpu()
    chan = g.dim() == 4
    a = g.exp() if chan else g.exp()[..., None]
    b = torch.ones(T, B, H, 1, dtype=torch.float64) if beta is None else beta.double().cpu()[..., None]
    h0 = torch.zeros(B, H, d, dtype=torch.float64) if h0 is None else h0.double().cpu()
    n = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    live = (torch.arange(T)[:, None] < n[None, :])[..., None, None]
    a, x = torch.where(live, a, 1.0), torch.where(live, b * v, 0.0)
    h = run_recurrence(a, x, h0)
    S = run_recurrence(a, x.abs(), h0.abs())
    R = run_recurrence(a, S, torch.zeros_like(h0))
    err = C_SCAN * U * R
    last = lambda y, z: y[-1] if T else z  # noqa: E731
    res = {"out": (h * live, err * live), "h_last": (last(h, h0), last(err, torch.zeros_like(h0)))}
    if grad_last is None and grad_out is None:
        return res
    dy = torch.zeros_like(x) if grad_out is None else torch.where(live, grad_out.double().cpu(), 0.0)
    X0 = torch.zeros_like(h0) if grad_last is None else grad_last.double().cpu()
    # reversed time: e_t = a_{t+1} e_{t+1} + dy_t, with grad_last entering at the end
    later = torch.cat([a[1:], torch.ones_like(a[:1])]).flip(0)
    D = run_recurrence(later, dy.flip(0), X0).flip(0)
    SD = run_recurrence(later, dy.abs().flip(0), X0.abs())
    RD = C_SCAN * U * run_recurrence(later, SD, torch.zeros_like(h0)).flip(0)
    before = torch.cat([h0[None], h])[:T]
    err_before = torch.cat([torch.zeros_like(h0)[None], err])[:T]
    res["grad_v"] = (b * D * live, b.abs() * (RD + 2 * U * D.abs()) * live)
    gg = a * before * D * live
    eg = a * (err_before * D.abs() + before.abs() * RD + 16 * U * before.abs() * D.abs()) * live
    res["grad_g"] = (gg, eg) if chan else (gg.sum(-1), eg.sum(-1))
    if beta is not None:
        res["grad_beta"] = ((v * D * live).sum(-1), (v.abs() * (RD + 16 * U * D.abs()) * live).sum(-1))
    res["grad_h0"] = ((a[0] * D[0], a[0] * (RD[0] + 8 * U * D[0].abs())) if T else (X0, torch.zeros_like(X0)))
    return res


def turned(u, positions, inv_freq, pairs, back=False):
    """u [M, heads, d] with its first 2 len(inv_freq) channels turned, and the sums of absolute values in its terms."""
    if inv_freq is None:
        return u, u.abs()
    r = 2 * inv_freq.numel()
    angle = positions.double().cpu().reshape(-1)[:, None, None] * inv_freq.double().cpu()
    c, s = angle.cos(), -angle.sin() if back else angle.sin()
    i = torch.arange(r // 2)
    first, second = (i, i + r // 2) if pairs == "half" else (2 * i, 2 * i + 1)
    y, size = u.clone(), u.abs()
    a, b = u[..., first], u[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = a.abs() + b.abs()
    return y, size


def qk(x, positions, inv_freq, weight, norm, eps, pairs, scale, grad=None):
    """One of q and k [M, heads, d]: {name: (value, bound)} in FP64 on the CPU."""
    x = x.double().cpu()
    d = x.shape[-1]
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double().cpu()
    n = (x * x).sum(-1, keepdim=True)
    r = ((n if norm == "l2" else n / d) + eps) ** -0.5
    xh = x * r
    y, size = turned(xh * w, positions, inv_freq, pairs)
    res = {"y": (y * scale, C_QK * U * abs(scale) * size)}
    if grad is None:
        return res
    dz, size = turned(grad.double().cpu() * scale, positions, inv_freq, pairs, back=True)
    M = x.shape[0] * x.shape[1]
    res["dw"] = ((dz * xh).sum((0, 1)), (2 * C_QK + M) * U * (size * xh.abs()).sum((0, 1)))
    du, size = dz * w, size * w.abs()
    k = 1.0 if norm == "l2" else 1.0 / d
    c = (xh * du).sum(-1, keepdim=True) * k
    c_size = (xh.abs() * size).sum(-1, keepdim=True) * k
    res["dx"] = (r * (du - xh * c), 3 * C_QK * U * r * (size + xh.abs() * c_size))
    return res


def check(got, want, dtype=torch.float32, what=""):
    """|got - value| <= bound + half a step of the type (an output is rounded once)."""
    value, bound = want
    got = got.detach().double().cpu().reshape(value.shape)
    lim = bound + step(dtype) * (value.abs() + bound) + 1e-38
    off = (got - value).abs()
    assert torch.isfinite(got).all() or not torch.isfinite(value).all(), what
    bad = off > lim
    if bad.any():
        i = int((off / lim).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / lim).max()):.3g} of its "
                             f"bound at {i}: got {float(got.reshape(-1)[i])}, want {float(value.reshape(-1)[i])}")
