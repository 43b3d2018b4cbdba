"""The gated scan and its gradients against the 64-bit recurrence, at the sizes,
layouts and masks where a split sequence can go wrong."""
import pytest
import torch

import plain_ops
from recurrent_state_quantization_lq_b200 import lq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def case(T, B, H, d, chan=False, dtype=BF, beta=True, ragged=False, order="token", seed=0, slow=0.03):
    """Inputs as a layer gives them, with heads that forget slowly (slow) and at once."""
    gen = torch.Generator().manual_seed(seed)
    lead = (T, B, H) if order == "token" else (B, T, H)
    laid = (lambda x: x) if order == "token" else (lambda x: x.transpose(0, 1))
    on = lambda x: laid(x.to(DEV))  # noqa: E731
    c = {"v": on(torch.randn(*lead, d, generator=gen).to(dtype))}
    g = torch.randn(*lead, *([d] if chan else []), generator=gen)
    c["g"] = on(-slow * torch.nn.functional.softplus(g) * (1 + 20 * (torch.arange(H) % 2)).reshape(
        (H, 1) if chan else (H,)))
    c["beta"] = on(torch.sigmoid(torch.randn(*lead, generator=gen))) if beta else None
    c["h0"] = torch.randn(B, H, d, generator=gen).to(DEV)
    c["grad_out"] = on(torch.randn(*lead, d, generator=gen).to(dtype))
    c["grad_last"] = torch.randn(B, H, d, generator=gen).to(DEV)
    c["lengths"] = None
    if ragged:
        n = torch.randint(0, T + 1, (B,), generator=gen, dtype=torch.int32)
        n[0], n[-1] = T, 0
        c["lengths"] = n.to(DEV)
    return c


def run(c, **kw):
    marks = lq.gated_scan_checkpoints(c["v"], c["g"])
    marks.fill_(float("nan"))
    out, last = lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"], lengths=c["lengths"], checkpoints=marks, **kw)
    gv, gg, gb, gh = lq.gated_scan_backward(c["grad_out"].to(out.dtype), c["v"], c["g"], c["beta"],
                                            checkpoints=marks, grad_last=c["grad_last"], lengths=c["lengths"])
    return {"out": out, "h_last": last, "grad_v": gv, "grad_g": gg, "grad_beta": gb, "grad_h0": gh}


def verify(c, got):
    want = plain_ops.scan(c["v"], c["g"], c["beta"], c["h0"], c["lengths"], c["grad_out"].to(got["out"].dtype),
                          c["grad_last"])
    for name, w in want.items():
        plain_ops.check(got[name], w, got[name].dtype, name)
    assert ("grad_beta" in want) == (got["grad_beta"] is not None)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 15, 31, 33, 63, 64, 65, 127, 129, 257, 511, 1000, 2049])
def test_lengths_of_one_sequence(T):
    c = case(T, 1, 3, 64, seed=T)
    verify(c, run(c))


@pytest.mark.parametrize("d", [1, 2, 3, 7, 8, 9, 12, 16, 31, 40, 64, 72, 96, 100, 127, 128, 136, 200, 255, 256])
@pytest.mark.parametrize("chan", [False, True])
def test_channels(d, chan):
    c = case(150, 2, 3, d, chan=chan, dtype=F32 if d % 3 == 0 else BF, seed=d)
    verify(c, run(c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("chan", [False, True])
@pytest.mark.parametrize("order", ["token", "sequence"])
@pytest.mark.parametrize("beta", [False, True])
def test_types_gates_and_orders(dtype, out_dtype, chan, order, beta):
    c = case(333, 2, 4, 128, chan=chan, dtype=dtype, order=order, beta=beta, ragged=True, seed=5)
    verify(c, run(c, out_dtype=out_dtype))


@pytest.mark.parametrize("T,B,H,d", [(700, 5, 2, 64), (2500, 3, 1, 128), (40, 70, 8, 32), (9, 4, 4, 100)])
def test_ragged_batches(T, B, H, d):
    c = case(T, B, H, d, ragged=True, seed=T)
    verify(c, run(c))


@pytest.mark.parametrize("B,H", [(1, 1), (1, 160), (37, 9)])
def test_few_and_many_heads(B, H):
    c = case(600, B, H, 32, chan=True, seed=B)
    verify(c, run(c))


def test_rows_past_a_length_are_neither_read_nor_written():
    T, B, H, d = 300, 4, 3, 64
    c = case(T, B, H, d, seed=3)
    c["lengths"] = torch.tensor([0, 1, 130, 300], dtype=torch.int32, device=DEV)
    past = (torch.arange(T, device=DEV)[:, None] >= c["lengths"][None, :])
    for name in ("v", "g", "beta", "grad_out"):
        c[name][past] = float("nan")
    marks = lq.gated_scan_checkpoints(c["v"], c["g"])
    out = torch.full((T, B, H, d), 7.0, dtype=BF, device=DEV)
    res, last = lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"], lengths=c["lengths"], out=out, checkpoints=marks)
    assert res is out and (out[past] == 7).all() and torch.isfinite(out).all() and torch.isfinite(last).all()
    gv, gg, gb = (torch.full_like(c[n], 7.0) for n in ("v", "g", "beta"))
    _, _, _, gh = lq.gated_scan_backward(c["grad_out"], c["v"], c["g"], c["beta"], checkpoints=marks,
                                         grad_last=c["grad_last"], lengths=c["lengths"], grad_v=gv, grad_g=gg,
                                         grad_beta=gb)
    for x in (gv, gg, gb):
        assert (x[past] == 7).all() and torch.isfinite(x).all()
    assert torch.equal(gh[0], c["grad_last"][0])          # no token: the gradient passes through
    assert torch.equal(last[0], c["h0"][0])


def test_lengths_out_of_range_are_clamped():
    c = case(50, 2, 2, 64, seed=8)
    c["lengths"] = torch.tensor([-5, 1000], dtype=torch.int32, device=DEV)
    verify(c, run(c))


def test_no_tokens():
    c = case(0, 2, 3, 64)
    out, last = lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"])
    assert out.numel() == 0 and torch.equal(last, c["h0"])
    _, last = lq.gated_scan(c["v"], c["g"])
    assert (last == 0).all()
    gh = lq.gated_scan_backward(c["grad_out"], c["v"], c["g"], c["beta"], grad_last=c["grad_last"],
                                checkpoints=lq.gated_scan_checkpoints(c["v"], c["g"]))[3]
    assert torch.equal(gh, c["grad_last"])


@pytest.mark.parametrize("chan", [False, True])
def test_gates_that_close_and_extreme_values(chan):
    """-inf empties the state, 0 keeps it, and an infinity or NaN stays in its channel and time."""
    T, B, H, d = 200, 1, 2, 64
    c = case(T, B, H, d, chan=chan, dtype=F32, seed=2)
    c["g"][17], c["g"][130] = float("-inf"), 0.0
    c["g"][40] = -200.0                       # exp underflows to zero
    verify(c, run(c))
    c["v"][60, 0, 0, 5] = float("inf")
    c["v"][61, 0, 0, 9] = float("nan")
    out, last = lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"])
    assert torch.isfinite(out[:60]).all() and torch.isfinite(out[:, :, 1]).all()
    assert torch.isinf(out[60:, 0, 0, 5]).all() and torch.isnan(out[61:, 0, 0, 9]).all()
    others = [i for i in range(d) if i not in (5, 9)]
    assert torch.isfinite(out[:, 0, 0, others]).all() and torch.isnan(last[0, 0, 9])


def test_strided_and_offset_views():
    """Views into wider tensors, unaligned starts and an expanded gate give what packed copies give."""
    T, B, H, d = 130, 2, 3, 64
    c = case(T, B, H, d, seed=11)
    want = run(c)
    wide = torch.randn(T, B, H, 3 * d + 1, device=DEV).to(BF)
    for off in (0, 64, 5):                    # aligned rows are impossible here: 193 channels apart
        wide[..., off:off + d] = c["v"]
        got = run({**c, "v": wide[..., off:off + d]})
        for n, x in got.items():
            assert torch.equal(x, want[n]), (off, n)
    even = torch.zeros(T, B, H, 2 * d, dtype=BF, device=DEV)
    even[..., d:] = c["v"]
    got = run({**c, "v": even[..., d:]})
    for n, x in got.items():
        assert torch.equal(x, want[n]), n
    one = c["g"][:, :, :1].expand(T, B, H)
    got = run({**c, "g": one})
    verify({**c, "g": one}, got)


def test_state_in_place_and_tokens_one_by_one():
    """Decoding token by token in place follows the scan over all of them."""
    T, B, H, d = 70, 3, 2, 128
    c = case(T, B, H, d, seed=4)
    want = plain_ops.scan(c["v"], c["g"], c["beta"], c["h0"], None)
    h = c["h0"].clone()
    for t in range(T):
        out, last = lq.gated_scan(c["v"][t:t + 1], c["g"][t:t + 1], c["beta"][t:t + 1], h, h_last=h)
        assert last is h
        plain_ops.check(out[0], tuple(x[t] for x in want["out"]), BF, f"token {t}")
    plain_ops.check(h, want["h_last"], F32, "h_last")


@pytest.mark.parametrize("T", [40, 900, 5000])
def test_state_and_gradient_in_place_over_a_cluster(T):
    """h_last may be h0 and grad_h0 grad_last also where several CTAs read them."""
    c = case(T, 1, 2, 128, seed=T)
    want = run(c)
    for _ in range(5):
        h, dh = c["h0"].clone(), c["grad_last"].clone()
        marks = lq.gated_scan_checkpoints(c["v"], c["g"])
        out, last = lq.gated_scan(c["v"], c["g"], c["beta"], h, h_last=h, checkpoints=marks)
        gh = lq.gated_scan_backward(c["grad_out"], c["v"], c["g"], c["beta"], checkpoints=marks, grad_last=dh,
                                    grad_h0=dh)[3]
        assert last is h and gh is dh and torch.equal(out, want["out"])
        assert torch.equal(h, want["h_last"]) and torch.equal(dh, want["grad_h0"])


@pytest.mark.parametrize("T", [6, 18, 40, 64, 65])
def test_few_tokens_of_many_heads(T):
    """On both sides of the token-by-token kernel's rule, with its checkpoints."""
    c = case(T, 40, 32, 64, seed=T, ragged=True)
    verify(c, run(c))


def test_two_calls_at_once():
    """Two streams run the same operator on their own data."""
    cs = [case(3000, 2, 8, 128, seed=s) for s in (1, 2)]
    want = [run(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(4):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                got[i].append(run(c))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for n in r:
                assert torch.equal(r[n], want[i][n]), n


def test_a_split_prompt_continues():
    c = case(900, 2, 2, 64, seed=6)
    whole, last = lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"], out_dtype=F32)
    cut = 333
    first, h = lq.gated_scan(c["v"][:cut], c["g"][:cut], c["beta"][:cut], c["h0"], out_dtype=F32)
    rest, h = lq.gated_scan(c["v"][cut:], c["g"][cut:], c["beta"][cut:], h, out_dtype=F32)
    want = plain_ops.scan(c["v"], c["g"], c["beta"], c["h0"], None)
    plain_ops.check(torch.cat([first, rest]), want["out"], F32)
    plain_ops.check(h, want["h_last"], F32)
    plain_ops.check(whole, want["out"], F32)
    none, h2 = lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"], want_out=False)
    assert none is None and torch.equal(h2, last)


def test_runs_are_equal_bit_for_bit():
    c = case(1500, 2, 4, 128, ragged=True, seed=9)
    a, b = run(c), run(c)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_a_gradient_of_the_outputs_alone_and_of_the_state_alone():
    c = case(140, 2, 2, 64, seed=13)
    marks = lq.gated_scan_checkpoints(c["v"], c["g"])
    lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"], checkpoints=marks)
    for dy, dh in ((c["grad_out"], None), (None, c["grad_last"])):
        got = lq.gated_scan_backward(dy, c["v"], c["g"], c["beta"], checkpoints=marks, grad_last=dh)
        want = plain_ops.scan(c["v"], c["g"], c["beta"], c["h0"], None, dy, dh)
        for x, n in zip(got, ("grad_v", "grad_g", "grad_beta", "grad_h0")):
            plain_ops.check(x, want[n], x.dtype, n)


def test_gradients_follow_differences():
    """The loss sum(out W) + sum(h_last w) is linear in v, in beta and in h0, so a finite difference
    of the kernel's own outputs equals the gradient's product with the direction up to rounding;
    along g the 64-bit reference is differenced."""
    T, B, H, d = 90, 1, 2, 32
    c = case(T, B, H, d, dtype=F32, seed=21)
    got = run(c)

    def loss(**kw):
        x = {**c, **kw}
        out, last = lq.gated_scan(x["v"], x["g"], x["beta"], x["h0"])
        return float((out.double() * c["grad_out"].double()).sum() + (last.double() * c["grad_last"].double()).sum())

    def loss64(g):
        r = plain_ops.scan(c["v"], g, c["beta"], c["h0"], None)
        return float((r["out"][0] * c["grad_out"].double().cpu()).sum() +
                     (r["h_last"][0] * c["grad_last"].double().cpu()).sum())

    r = plain_ops.scan(c["v"], c["g"], c["beta"], c["h0"], None)
    noise = float((r["out"][1] * c["grad_out"].double().cpu().abs()).sum() +
                  (r["h_last"][1] * c["grad_last"].double().cpu().abs()).sum())
    for name in ("v", "beta", "h0"):
        gen = torch.Generator().manual_seed(1)
        way = torch.randn(c[name].shape, generator=gen).to(DEV)
        diff = loss(**{name: c[name] + way}) - loss(**{name: c[name] - way})
        slope = 2 * float((got["grad_" + name].double() * way.double()).sum())
        # the perturbed runs are at most 5 times as large as this one; rounding c + way adds a u
        assert abs(diff - slope) <= 12 * noise + 1e-5 * abs(slope), (name, diff, slope)
    gen = torch.Generator().manual_seed(2)
    way = torch.randn(c["g"].shape, generator=gen, dtype=torch.float64)
    e = 1e-5
    g64 = c["g"].double().cpu()
    diff = (loss64(g64 + e * way) - loss64(g64 - e * way)) / (2 * e)
    slope = float((got["grad_g"].double().cpu() * way).sum())
    want = plain_ops.scan(c["v"], c["g"], c["beta"], c["h0"], None, c["grad_out"], c["grad_last"])["grad_g"]
    # the difference's own error: third derivatives times e^2 / 6, below 1e-6 of the slopes' absolute sum
    lim = float((want[1] * way.abs()).sum()) + 1e-6 * float((want[0] * way).abs().sum())
    assert abs(diff - slope) <= lim, (diff, slope)


def test_other_streams_and_graphs():
    c = case(500, 2, 4, 64, seed=15)
    want = run(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = {}
    marks = lq.gated_scan_checkpoints(c["v"], c["g"])
    got["out"], got["h_last"] = lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"], checkpoints=marks, stream=s)
    got["grad_v"], got["grad_g"], got["grad_beta"], got["grad_h0"] = lq.gated_scan_backward(
        c["grad_out"], c["v"], c["g"], c["beta"], checkpoints=marks, grad_last=c["grad_last"], stream=s)
    s.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
    static = {n: x.clone() for n, x in c.items() if x is not None} | {"lengths": None}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = run(static)
    other = case(500, 2, 4, 64, seed=16)
    for n, x in other.items():
        if x is not None:
            static[n].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    want = run(other)
    for n in want:
        assert torch.equal(res[n], want[n]), n


def test_offsets_past_32_bits():
    """A token stride that puts the last token more than 2^31 elements away."""
    T, B, H, d = 5, 1, 1, 64
    c = case(T, B, H, d, seed=17)
    far = (1 << 29) + 64
    store = torch.empty(far * (T - 1) + d, dtype=BF, device=DEV)
    v = store.as_strided((T, B, H, d), (far, d, d, 1))
    v.copy_(c["v"])
    want, got = run(c), run({**c, "v": v})
    for n in want:
        assert torch.equal(got[n], want[n]), n
