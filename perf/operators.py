"""The gated scan and the q/k norm with rotation: their plain forms, and calls to measure.

`run` computes either the plain form (elementary torch operations in FP32) or,
where `own` is true, makes the framework's calls.

Gated scan, for every (sequence, head, channel), a_t = exp(g_t):
    h_t = a_t h_{t-1} + beta_t v_t,  out_t = h_t
and its gradients.  q/k norm: every head's row is normalised (L2 or RMS,
optional weight), then its first rot_dim channels are rotated by the angles
position * inv_freq, then q is scaled.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
#: elements of the largest case; a drawn one has at most a quarter of them
MOST = 8192 * 8 * 32 * 128


def scan(name, T, B, H, d, gate="scalar", dtype="bf16", train=False, ragged=False, beta=True, order="token"):
    return {"name": name, "op": "scan", "T": T, "B": B, "H": H, "d": d, "gate": gate, "dtype": dtype, "train": train,
            "ragged": ragged, "beta": beta, "order": order}


def qk(name, M, hq, hk, d, norm="rms", rot=0, pairs="half", dtype="bf16", weights=True, train=False, fused=False,
       far=4096):
    return {"name": name, "op": "qk", "M": M, "hq": hq, "hk": hk, "d": d, "norm": norm, "rot": rot, "pairs": pairs,
            "dtype": dtype, "weights": weights, "train": train, "fused": fused, "far": far}


def listed():
    return [
        # one decode token of a full batch (64 sequences x 32 heads x 128): latency
        scan("scan_decode", 1, 64, 32, 128),
        # prompts of a ragged batch, up to 512 tokens, padded
        scan("scan_prompts_ragged", 512, 64, 32, 128, ragged=True),
        # one long document, sequence-major as a projection leaves it
        scan("scan_long_document", 65536, 1, 32, 128, order="sequence"),
        # a small training step at odd sizes in FP32, without an input gate
        scan("scan_train_odd", 1000, 3, 5, 100, gate="channel", dtype="f32", train=True, beta=False),
        # a training step of a layer with a gate for each channel
        scan("scan_train_channel", 4096, 4, 32, 128, gate="channel", train=True, order="sequence"),
        # the largest training step: 8 sequences of 8192 tokens
        scan("scan_train_large", 8192, 8, 32, 128, train=True),
        # q and k of one decode token of a full batch, L2-normalised: latency
        qk("qk_decode", 64, 32, 32, 128, norm="l2", weights=False),
        # one decode token of a small batch with grouped keys, rotated, cut out of a fused projection
        qk("qk_decode_rotated", 8, 32, 8, 128, rot=128, fused=True, far=1000000),
        # the prompts of a batch: 64 x 512 tokens
        qk("qk_prompts", 32768, 32, 8, 128, rot=128, fused=True),
        # a training step, half of the channels rotated
        qk("qk_train", 16384, 32, 8, 128, rot=64, train=True),
        # a training step at odd sizes in FP32, neighbouring pairs, far positions
        qk("qk_train_odd", 1111, 6, 3, 80, rot=48, pairs="neighbours", dtype="f32", train=True, far=1000000),
        # L2-normalised and rotated small heads, training
        qk("qk_train_l2", 8192, 32, 32, 64, norm="l2", rot=64, weights=False, train=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            c = scan("", _log(rng, 1, 65536), _log(rng, 1, 64), _log(rng, 1, 48),
                     rng.choice([64, 128, 256, _log(rng, 8, 256)]), rng.choice(["scalar", "channel"]),
                     rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.7,
                     rng.choice(["token", "sequence"]))
            if 1000 <= c["T"] * c["B"] * c["H"] * c["d"] <= MOST // 4:
                break
    else:
        while True:
            d = rng.choice([64, 128, 256, 2 * _log(rng, 4, 128)])
            hk = _log(rng, 1, 32)
            c = qk("", _log(rng, 1, 65536), hk * rng.choice([1, 2, 4]), hk, d, rng.choice(["rms", "l2"]),
                   rng.choice([0, d, d, 2 * rng.randint(1, d // 2)]), rng.choice(["half", "neighbours"]),
                   rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.6, rng.random() < 0.5, rng.random() < 0.4,
                   rng.choice([4096, 1000000]))
            if c["M"] * (c["hq"] + c["hk"]) * d <= MOST // 4:
                break
    del c["name"]
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "scan":
        T, B, H, d = case["T"], case["B"], case["H"], case["d"]
        lead = (B, T, H) if case["order"] == "sequence" else (T, B, H)

        def laid(x):  # token-major views, whatever the order in memory
            return x.transpose(0, 1) if case["order"] == "sequence" else x

        s["v"] = laid(normal(*lead, d, dtype=dt))
        g = normal(*lead, d) if case["gate"] == "channel" else normal(*lead)
        # heads that forget within ten tokens up to ones that remember a thousand
        keep = torch.pow(10.0, -2 * torch.rand(H, generator=gen, device="cuda")).mul_(-0.1)
        s["g"] = laid(torch.nn.functional.softplus(g).mul_(keep[:, None] if case["gate"] == "channel" else keep))
        s["beta"] = laid(torch.sigmoid(normal(*lead))) if case["beta"] else None
        s["h0"] = normal(B, H, d)
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        if case["train"]:
            s["grad_out"] = laid(normal(*lead, d, dtype=dt))
            s["grad_last"] = normal(B, H, d)
        return s
    M, hq, hk, d = case["M"], case["hq"], case["hk"], case["d"]
    if case["fused"]:  # views into one projection's rows: q, k and as many values as keys
        x = normal(M, (hq + 2 * hk) * d, dtype=dt)
        s["q"], s["k"] = x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    else:
        s["q"], s["k"] = normal(M, hq, d, dtype=dt), normal(M, hk, d, dtype=dt)
    s["positions"] = s["inv_freq"] = s["weight_q"] = s["weight_k"] = None
    if case["rot"]:
        s["positions"] = torch.randint(0, case["far"], (M,), generator=gen, device="cuda", dtype=torch.int32)
        i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = torch.pow(10000.0, -2.0 * i / case["rot"])
    if case["weights"]:
        s["weight_q"], s["weight_k"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
    s["q_scale"] = d ** -0.5
    if case["train"]:
        s["grad_q"], s["grad_k"] = normal(M, hq, d, dtype=dt), normal(M, hk, d, dtype=dt)
    return s


# ------------------------------------------------------------------ the framework's calls
def run_own(s):
    from recurrent_state_quantization_lq_b200 import lq
    case = s["case"]
    if case["op"] == "scan":
        if not case["train"]:
            out, last = lq.gated_scan(s["v"], s["g"], s["beta"], s["h0"], lengths=s["lengths"])
            return {"out": out, "h_last": last}
        marks = lq.gated_scan_checkpoints(s["v"], s["g"])
        out, last = lq.gated_scan(s["v"], s["g"], s["beta"], s["h0"], lengths=s["lengths"], checkpoints=marks)
        gv, gg, gb, gh = lq.gated_scan_backward(s["grad_out"], s["v"], s["g"], s["beta"], checkpoints=marks,
                                                grad_last=s["grad_last"], lengths=s["lengths"])
        return {"out": out, "h_last": last, "grad_v": gv, "grad_g": gg, "grad_beta": gb, "grad_h0": gh}
    how = {"positions": s["positions"], "inv_freq": s["inv_freq"], "weight_q": s["weight_q"],
           "weight_k": s["weight_k"], "norm": case["norm"], "eps": EPS, "pairs": case["pairs"],
           "q_scale": s["q_scale"]}
    q, k = lq.qk_norm_rotate(s["q"], s["k"], **how)
    if not case["train"]:
        return {"q": q, "k": k}
    gq, gk, gwq, gwk = lq.qk_norm_rotate_backward(s["grad_q"], s["grad_k"], s["q"], s["k"], **how)
    return {"q": q, "k": k, "grad_q": gq, "grad_k": gk, "grad_weight_q": gwq, "grad_weight_k": gwk}


# ------------------------------------------------------------------ the plain forms
def _doubling(a, x):
    """h_t = a_t h_{t-1} + x_t over the first axis from zero, by doubling the run that each entry covers; in place."""
    step = 1
    while step < x.shape[0]:
        x[step:] += a[step:] * x[:-step]
        if 2 * step < x.shape[0]:
            a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return x


def plain_scan(s):
    case = s["case"]
    T, B, dt = case["T"], case["B"], s["v"].dtype
    a = torch.exp(s["g"].double()).float()  # in 64 bits: a gate near 1 acts over a thousand tokens
    a = a if case["gate"] == "channel" else a[..., None]
    x = s["v"].float()
    x = x * s["beta"][..., None] if case["beta"] else x.clone()
    live = None
    if case["ragged"]:  # a token past its sequence's length leaves the state as it is
        live = (torch.arange(T, device=a.device)[:, None] < s["lengths"][None, :])[..., None, None]
        a, x = torch.where(live, a, 1.0), torch.where(live, x, 0.0)
    x[0] += a[0] * s["h0"]
    h = _doubling(a, x)
    out = h if live is None else torch.where(live, h, 0.0)
    res = {"out": out.to(dt), "h_last": h[-1].clone()}
    if not case["train"]:
        return res
    dy = s["grad_out"].float()
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    later = torch.cat([torch.ones_like(a[:1]), a[1:].flip(0)])  # reversed time: the gate of the token after
    dy = dy.flip(0)
    dy[0] += s["grad_last"]
    D = _doubling(later, dy).flip(0)
    before = torch.cat([s["h0"][None], h[:-1]])
    gv = D * s["beta"][..., None] if case["beta"] else D
    gg = a * before * D
    gg = gg if case["gate"] == "channel" else gg.sum(-1)
    gb = (s["v"].float() * D).sum(-1) if case["beta"] else None
    if live is not None:
        gv = torch.where(live, gv, 0.0)
        gg = torch.where(live if case["gate"] == "channel" else live[..., 0], gg, 0.0)
        gb = torch.where(live[..., 0], gb, 0.0) if case["beta"] else None
    return {**res, "grad_v": gv.to(dt), "grad_g": gg, "grad_beta": gb, "grad_h0": a[0] * D[0]}


def _rotate(u, cos, sin, case):
    """Rotate the pairs of the first rot channels of u [M, heads, d]."""
    r = case["rot"]
    if not r:
        return u
    cos, sin = cos[:, None], sin[:, None]
    y = u.clone()
    first, second = (slice(0, r // 2), slice(r // 2, r)) if case["pairs"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    y[..., first] = u[..., first] * cos - u[..., second] * sin
    y[..., second] = u[..., second] * cos + u[..., first] * sin
    return y


def _plain_heads(x, dy, w, scale, cos, sin, case):
    """One of q and k: its output and, with dy, the gradients of its input and weight."""
    xf = x.float()
    n = (xf * xf).sum(-1, keepdim=True)
    r = torch.rsqrt((n if case["norm"] == "l2" else n / case["d"]) + EPS)
    xh = xf * r
    y = (_rotate(xh if w is None else xh * w, cos, sin, case) * scale).to(x.dtype)
    if dy is None:
        return y, None, None
    dz = _rotate(dy.float() * scale, cos, None if sin is None else -sin, case)
    gw = None if w is None else (dz * xh).sum((0, 1), dtype=torch.float64).float()
    du = dz if w is None else dz * w
    c = (xh * du).sum(-1, keepdim=True)
    return y, (r * (du - xh * (c if case["norm"] == "l2" else c / case["d"]))).to(x.dtype), gw


def plain_qk(s):
    case = s["case"]
    cos = sin = None
    if case["rot"]:  # far positions: the angles in 64 bits
        angle = s["positions"].double()[:, None] * s["inv_freq"]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q, gq, gwq = _plain_heads(s["q"], s.get("grad_q"), s["weight_q"], s["q_scale"], cos, sin, case)
    k, gk, gwk = _plain_heads(s["k"], s.get("grad_k"), s["weight_k"], 1.0, cos, sin, case)
    if not case["train"]:
        return {"q": q, "k": k}
    return {"q": q, "k": k, "grad_q": gq, "grad_k": gk, "grad_weight_q": gwq, "grad_weight_k": gwk}


def run(state):
    if own:
        return run_own(state)
    return plain_scan(state) if state["case"]["op"] == "scan" else plain_qk(state)


# ------------------------------------------------------------------ work and exact values
def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "scan":
        T, n = case["T"], case["B"] * case["H"]
        if case["ragged"]:
            T = T / 2  # lengths are uniform over 0..T
        rows, states = T * n, 4 * n * case["d"]
        gate = 4 * (case["d"] if case["gate"] == "channel" else 1) + (4 if case["beta"] else 0)
        row = 2 * e * case["d"] + gate                     # v in, out; g and beta in
        if case["train"]:
            row += 2 * e * case["d"] + gate                # grad_out in, grad_v; grad_g and grad_beta
        return {"bytes": rows * row + states * (4 if case["train"] else 2),
                "flops": rows * case["d"] * (14 if case["train"] else 3)}
    x = case["M"] * (case["hq"] + case["hk"]) * case["d"]
    return {"bytes": x * e * (4 if case["train"] else 2) + (4 * case["M"] if case["rot"] else 0),
            "flops": x * (24 if case["train"] else 9)}


def exact(case, seed):
    """The definitions in 64 bits: the recurrence one token after another, the norms by differentiating their formula."""
    s = prepare(case, seed)
    if case["op"] == "scan":
        return _exact_scan(case, s)
    res = {}
    for n, scale in (("q", s["q_scale"]), ("k", 1.0)):
        x = s[n].double().detach().requires_grad_(case["train"])
        w = torch.ones(case["d"], device=x.device, dtype=torch.float64)
        w = (w if s["weight_" + n] is None else s["weight_" + n].double()).requires_grad_(case["train"])
        size = x.square().sum(-1, keepdim=True) if case["norm"] == "l2" else x.square().mean(-1, keepdim=True)
        u = x / torch.sqrt(size + EPS) * w * scale
        r = case["rot"]
        if r:
            turn = torch.polar(torch.ones((), device=x.device, dtype=torch.float64),
                               s["positions"].double()[:, None, None] * s["inv_freq"])
            if case["pairs"] == "half":
                z = torch.complex(u[..., :r // 2], u[..., r // 2:r]) * turn
                y = torch.cat([z.real, z.imag, u[..., r:]], -1)
            else:
                z = torch.view_as_complex(u[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * turn
                y = torch.cat([torch.view_as_real(z).flatten(-2), u[..., r:]], -1)
        else:
            y = u
        if case["train"]:
            gx, gw = torch.autograd.grad(y, (x, w), s["grad_" + n].double())
            res["grad_" + n], res["grad_weight_" + n] = gx, gw if case["weights"] else None
        res[n] = y.detach()
    return res


def _exact_scan(case, s):
    T = case["T"]
    a = s["g"].double().exp()
    a = a if case["gate"] == "channel" else a.unsqueeze(-1)
    v = s["v"].double()
    beta = s["beta"].double().unsqueeze(-1) if case["beta"] else torch.ones_like(v[..., :1])
    on = torch.ones(T, case["B"], 1, 1, device=v.device, dtype=torch.bool)
    if case["ragged"]:
        on = torch.arange(T, device=v.device).view(T, 1, 1, 1) < s["lengths"].view(1, -1, 1, 1)
    ragged, h, states = case["ragged"], s["h0"].double(), torch.empty(v.shape, device=v.device, dtype=torch.float64)
    x = v * beta
    for t in range(T):
        new = torch.addcmul(x[t], a[t], h)
        h = torch.where(on[t], new, h) if ragged else new
        states[t] = h
    del x
    res = {"out": states * on if ragged else states, "h_last": h}
    if not case["train"]:
        return res
    gv, gg, gb = torch.empty_like(v), torch.empty_like(s["g"], dtype=torch.float64), None
    if case["beta"]:
        gb = torch.empty_like(s["beta"], dtype=torch.float64)
    X, dy = s["grad_last"].double(), s["grad_out"].double()
    for t in range(T - 1, -1, -1):
        D = dy[t] + X
        new = a[t] * D
        if ragged:
            X, D, new = torch.where(on[t], new, X), D * on[t], new * on[t]
        else:
            X = new
        gv[t] = D
        slope = new * (states[t - 1] if t else s["h0"].double())
        gg[t] = slope if case["gate"] == "channel" else slope.sum(-1)
        if gb is not None:
            gb[t] = (v[t] * D).sum(-1)
    return {**res, "grad_v": gv.mul_(beta), "grad_g": gg, "grad_beta": gb, "grad_h0": X}
