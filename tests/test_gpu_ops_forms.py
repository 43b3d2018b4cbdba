"""Forms of the stateless operators that no other test runs: every compiled head size over clusters, mixed types,
rows of odd sizes over long sequences, calls at once, captured and replayed, on a given stream."""
import pytest
import torch

import plain_ops
import test_gpu_qk_norm as qk
import test_gpu_scan as scan
from recurrent_state_quantization_lq_b200 import lq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("chan", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,B,H", [(2100, 1, 2), (700, 5, 40)])
def test_compiled_head_sizes_with_and_without_clusters(d, chan, dtype, T, B, H):
    c = scan.case(T, B, H, d, chan=chan, dtype=dtype, ragged=B > 1, seed=d)
    scan.verify(c, scan.run(c))


@pytest.mark.parametrize("d", [1, 4, 8, 12, 24, 90, 96, 100, 192, 200, 250])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, F32), (F32, BF), (BF, BF)])
@pytest.mark.parametrize("chan", [False, True])
def test_other_head_sizes_and_mixed_types_over_clusters(d, dtype, out_dtype, chan):
    c = scan.case(1700, 2, 1, d, chan=chan, dtype=dtype, ragged=True, order="sequence", seed=d)
    scan.verify(c, scan.run(c, out_dtype=out_dtype))


def test_results_given_at_any_stride():
    """out and the gradients as views into wider tensors; what lies between their rows stays as it was."""
    T, B, H, d = 300, 2, 3, 64
    for wide, at in ((2 * d, 0), (2 * d, 8), (2 * d + 1, 1)):
        c = scan.case(T, B, H, d, ragged=True, seed=wide + at)
        want = scan.run(c)
        live = torch.arange(T, device=DEV)[:, None] < c["lengths"][None, :]
        marks = lq.gated_scan_checkpoints(c["v"], c["g"])
        hold = [torch.full((T, B, H, wide), 7.0, dtype=BF, device=DEV) for _ in range(2)]
        out, gv = (x[..., at:at + d] for x in hold)
        gg, gb = (torch.full((T, B, H, 2), 7.0, device=DEV) for _ in range(2))
        lq.gated_scan(c["v"], c["g"], c["beta"], c["h0"], lengths=c["lengths"], checkpoints=marks, out=out)
        lq.gated_scan_backward(c["grad_out"], c["v"], c["g"], c["beta"], checkpoints=marks, grad_last=c["grad_last"],
                               lengths=c["lengths"], grad_v=gv, grad_g=gg[..., 1], grad_beta=gb[..., 0])
        for x, n in ((out, "out"), (gv, "grad_v"), (gg[..., 1], "grad_g"), (gb[..., 0], "grad_beta")):
            assert torch.equal(x[live], want[n][live]) and (x[~live] == 7).all(), (n, wide)
        for x in hold:
            assert (x[..., :at] == 7).all() and (x[..., at + d:] == 7).all()
        assert (gg[..., 0] == 7).all() and (gb[..., 1] == 7).all()


def test_windows_over_a_sequence():
    """Tokens that overlap in memory (sliding windows): as their copies."""
    T, B, H, d = 500, 1, 2, 64
    c = scan.case(T, B, H, d, seed=3)
    for step in (8, 3):
        data = torch.randn(2 * (step * T + d), generator=torch.Generator().manual_seed(step)).to(BF).to(DEV)
        v = data.as_strided((T, B, H, d), (step, 0, step * T, 1))
        want, got = scan.run({**c, "v": v.contiguous()}), scan.run({**c, "v": v})
        for n in want:
            assert torch.equal(got[n], want[n]), (step, n)


@pytest.mark.parametrize("T", [1, 30, 2500])
def test_two_graphs_replayed_at_once(T):
    """Graphs captured one after the other share no memory that either writes."""
    cs = [scan.case(T, 3, 8, 128, seed=s) for s in (1, 2)]
    ns = [qk.case(257, 6, 2, 128, rot=128, seed=s) for s in (1, 2)]

    def call(c, n):
        return [*scan.run(c).values(), *lq.qk_norm_rotate(n[0]["q"], n[0]["k"], **n[1]),
                *lq.qk_norm_rotate_backward(n[0]["gq"], n[0]["gk"], n[0]["q"], n[0]["k"], **n[1])]

    want = [call(c, n) for c, n in zip(cs, ns)]
    torch.cuda.synchronize()
    graphs, got, streams = [], [], []
    for c, n in zip(cs, ns):
        graphs.append(torch.cuda.CUDAGraph())
        streams.append(torch.cuda.Stream())
        with torch.cuda.graph(graphs[-1]):
            got.append(call(c, n))
    for _ in range(5):
        for x in got[0] + got[1]:
            x.fill_(7.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_norms_at_once_on_two_streams():
    ns = [qk.case(9000, 8, 2, 64, rot=64, seed=s) for s in (3, 4)]
    call = lambda n, s=None: [*lq.qk_norm_rotate(n[0]["q"], n[0]["k"], stream=s, **n[1]),  # noqa: E731
                              *lq.qk_norm_rotate_backward(n[0]["gq"], n[0]["gk"], n[0]["q"], n[0]["k"], stream=s, **n[1])]
    want = [call(n) for n in ns]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ns]
    got = [[call(n, s) for _ in range(4)] for n, s in zip(ns, streams)]
    torch.cuda.synchronize()
    for runs, w in zip(got, want):
        assert all(torch.equal(x, y) for r in runs for x, y in zip(r, w))


def test_tokens_spread_over_heads_in_place():
    """Few tokens of many heads: a token's heads are taken in parts by several row groups, also in place."""
    for M, hq, hk, d, rot in ((1, 100, 7, 40, 40), (3, 64, 64, 8, 8), (2, 33, 1, 256, 200)):
        c, how = qk.case(M, hq, hk, d, rot=rot, seed=M)
        want, _ = qk.verify(c, how)
        q, k = c["q"].clone(), c["k"].clone()
        lq.qk_norm_rotate(q, k, q_out=q, k_out=k, **how)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("ragged", [False, True])
def test_a_state_with_norms_on_a_given_stream_and_in_a_graph(ragged):
    B, H, d, W = 3, 4, 64, 8
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(6, B, 3, H, d, generator=gen).to(BF).to(DEV)
    g = (-0.1 * torch.rand(6, B, H, generator=gen)).to(DEV)
    beta = torch.rand(6, B, H, generator=gen).to(DEV)
    how = {"inv_freq": 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device=DEV) / (d // 2))}
    v = x[:, :, 2].contiguous()
    pos = [torch.full((B,), t, dtype=torch.int32, device=DEV) for t in range(6)]
    outs = []
    for way in ("plain", "stream", "graph"):
        st = lq.DecodeState(B, H, d, window=W, ragged=ragged, device=DEV, qk_norm=how)
        st.prefill(None)
        o = torch.zeros(6, B, H, d, device=DEV)
        torch.cuda.synchronize()
        step = lambda t, s=None: st.decode_step(x[t, :, 0], x[t, :, 1], v[t], g[t], beta[t], out=o[t],  # noqa: E731
                                                positions=pos[t], stream=s)
        if way == "graph":
            step(0)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for t in range(1, 6):
                    step(t)
            graph.replay()
        else:
            s = torch.cuda.Stream() if way == "stream" else None
            for t in range(6):
                step(t, s)
        torch.cuda.synchronize()
        assert st.device_status() == lq.LQ_OK
        outs.append(o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and outs[0][5].abs().max() > 0
