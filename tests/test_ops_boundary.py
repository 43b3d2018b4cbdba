"""Refusals of the stateless operators, without a GPU: every call below returns before any launch."""
import ctypes

import pytest
import torch

from recurrent_state_quantization_lq_b200 import lq

P = 1 << 21                         # addresses that nothing reads
ref = ctypes.byref


def scan_config(**kw):
    return lq.ScanConfig(**{"batch": 2, "heads": 3, "d": 64, "gate": 0, "in_dtype": 1, "out_dtype": 1, **kw})


def scan_args(**kw):
    a = lq.ScanArgs(n_tokens=4, v=P, g=P, beta=P, h0=P, out=P, h_last=P, checkpoints=P, v_stride=(384, 192, 64),
                    g_stride=(6, 3, 1), beta_stride=(6, 3, 1), out_stride=(384, 192, 64))
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def scan_grads(**kw):
    g = lq.ScanGrads(grad_out=P, grad_last=P, grad_v=P, grad_g=P, grad_beta=P, grad_h0=P,
                     grad_out_stride=(384, 192, 64), grad_v_stride=(384, 192, 64), grad_g_stride=(6, 3, 1),
                     grad_beta_stride=(6, 3, 1))
    for n, x in kw.items():
        setattr(g, n, x)
    return g


@pytest.mark.parametrize("field,value", [("batch", 0), ("heads", 0), ("heads", 1 << 24), ("d", 0), ("d", 257), ("gate", 2),
                                         ("in_dtype", 2), ("out_dtype", -1)])
def test_scan_configs_refused(field, value):
    L, cfg = lq.lib(), scan_config(**{field: value})
    assert L.lq_gated_scan_checkpoint_bytes(ref(cfg), 4) == 0 and lq.last_error()
    assert L.lq_gated_scan(ref(cfg), ref(scan_args()), None) == lq.LQ_ERR_INVALID_ARG
    assert L.lq_gated_scan_backward(ref(cfg), ref(scan_args()), ref(scan_grads()), None) == lq.LQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,word", [({"n_tokens": -1}, "negative"), ({"n_tokens": (1 << 30) + 1}, "2^30"), ({"zero_past": 2}, "zero_past"), ({"v": None}, "NULL"),
                                     ({"g": None}, "NULL"), ({"v": P + 1}, "aligned"), ({"g": P + 2}, "aligned"),
                                     ({"lengths": P + 1}, "aligned"), ({"h0": P + 2}, "aligned"),
                                     ({"checkpoints": P + 3}, "aligned"), ({"beta": P + 1}, "aligned")])
def test_scan_arguments_refused(kw, word):
    L, cfg = lq.lib(), scan_config()
    assert L.lq_gated_scan(ref(cfg), ref(scan_args(**kw)), None) == lq.LQ_ERR_INVALID_ARG
    assert word in lq.last_error()
    assert L.lq_gated_scan_backward(ref(cfg), ref(scan_args(**kw)), ref(scan_grads()), None) == lq.LQ_ERR_INVALID_ARG
    assert word in lq.last_error()


def test_scan_outputs_and_gradients_refused():
    L, cfg = lq.lib(), scan_config()
    for kw in ({"out": P + 1}, {"h_last": P + 2}, {"out_stride": (0, 192, 64)}, {"out_stride": (384, 0, 64)},
               {"out_stride": (384, 192, 0)}):
        assert L.lq_gated_scan(ref(cfg), ref(scan_args(**kw)), None) == lq.LQ_ERR_INVALID_ARG, kw
    assert L.lq_gated_scan(ref(cfg), None, None) == lq.LQ_ERR_INVALID_ARG
    assert L.lq_gated_scan(None, ref(scan_args()), None) == lq.LQ_ERR_INVALID_ARG
    for kw in ({"grad_v": P + 1}, {"grad_g": P + 2}, {"grad_beta": P + 2}, {"grad_out": P + 1}, {"grad_last": P + 2},
               {"grad_h0": P + 2}, {"grad_v_stride": (0, 192, 64)}, {"grad_g_stride": (6, 3, 0)},
               {"grad_beta_stride": (6, 0, 1)}):
        assert L.lq_gated_scan_backward(ref(cfg), ref(scan_args()), ref(scan_grads(**kw)), None) == lq.LQ_ERR_INVALID_ARG, kw
    assert L.lq_gated_scan_backward(ref(cfg), ref(scan_args()), None, None) == lq.LQ_ERR_INVALID_ARG
    assert L.lq_gated_scan_backward(ref(cfg), ref(scan_args(checkpoints=None)), ref(scan_grads()), None) == lq.LQ_ERR_INVALID_ARG
    assert "checkpoints" in lq.last_error()
    assert L.lq_gated_scan_backward(ref(cfg), ref(scan_args(beta=None)), ref(scan_grads()), None) == lq.LQ_ERR_INVALID_ARG
    assert "grad_beta" in lq.last_error()


@pytest.mark.parametrize("d", [1, 8, 9, 64, 65, 128, 129, 256])
def test_checkpoints_are_small_and_grow_with_the_tokens(d):
    L, cfg = lq.lib(), scan_config(d=d)
    size = [L.lq_gated_scan_checkpoint_bytes(ref(cfg), n) for n in (0, 1, 32, 33, 4096, 1 << 20)]
    assert size[0] == 0 and size[1] == 6 * d * 4 and size == sorted(size)
    assert size[-1] <= -(-(1 << 20) // 24) * 6 * d * 4       # at least 24 tokens apart: 6 warps' rows of 4 tokens
    assert L.lq_gated_scan_checkpoint_bytes(ref(cfg), -1) == 0


def qk_config(**kw):
    return lq.QkNormConfig(**{"heads_q": 4, "heads_k": 2, "d": 64, "norm": 0, "rot_dim": 64, "pairs": 0, "dtype": 1,
                              "eps": 1e-6, "q_scale": 1.0, **kw})


def qk_args(**kw):
    return lq.QkNormArgs(**{"n_tokens": 5, "q": P, "k": P, "positions": P, "inv_freq": P, "weight_q": P, "weight_k": P,
                            "q_token": 256, "q_head": 64, "k_token": 128, "k_head": 64, **kw})


def pair(**kw):
    return lq.QkPair(**{"q": P, "k": P, "q_token": 256, "q_head": 64, "k_token": 128, "k_head": 64, **kw})


@pytest.mark.parametrize("kw", [{"heads_q": 0}, {"heads_k": -1}, {"d": 0}, {"d": 257}, {"norm": 2}, {"rot_dim": 63},
                                {"rot_dim": 66}, {"rot_dim": -2}, {"pairs": 2}, {"dtype": 3}, {"eps": 0.0}, {"eps": -1.0},
                                {"eps": float("nan")}, {"eps": float("inf")}, {"q_scale": float("inf")}])
def test_qk_configs_refused(kw):
    L, cfg = lq.lib(), qk_config(**kw)
    assert L.lq_qk_norm_rotate_workspace_bytes(ref(cfg)) == 0 and lq.last_error()
    assert L.lq_qk_norm_rotate(ref(cfg), ref(qk_args()), ref(pair()), None) == lq.LQ_ERR_INVALID_ARG
    assert L.lq_qk_norm_rotate_backward(ref(cfg), ref(qk_args()), ref(pair()), ref(pair()), P, P, P,
                                        None) == lq.LQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [{"n_tokens": -1}, {"n_tokens": 1 << 31}, {"q": None}, {"k": None}, {"positions": None},
                                {"inv_freq": None}, {"q": P + 1}, {"inv_freq": P + 4}, {"positions": P + 2},
                                {"weight_q": P + 2}])
def test_qk_arguments_refused(kw):
    L, cfg = lq.lib(), qk_config()
    assert L.lq_qk_norm_rotate(ref(cfg), ref(qk_args(**kw)), ref(pair()), None) == lq.LQ_ERR_INVALID_ARG
    assert L.lq_qk_norm_rotate_backward(ref(cfg), ref(qk_args(**kw)), ref(pair()), ref(pair()), None, None, None,
                                        None) == lq.LQ_ERR_INVALID_ARG


def test_qk_outputs_and_workspaces_refused():
    L, cfg = lq.lib(), qk_config()
    for kw in ({"q": None}, {"k": None}, {"q": P + 1}, {"q_token": 0}, {"k_head": 0}):
        assert L.lq_qk_norm_rotate(ref(cfg), ref(qk_args()), ref(pair(**kw)), None) == lq.LQ_ERR_INVALID_ARG, kw
        assert L.lq_qk_norm_rotate_backward(ref(cfg), ref(qk_args()), ref(pair()), ref(pair(**kw)), None, None, None,
                                            None) == lq.LQ_ERR_INVALID_ARG, kw
    back = L.lq_qk_norm_rotate_backward
    assert back(ref(cfg), ref(qk_args()), ref(pair()), ref(pair()), P, P, None, None) == lq.LQ_ERR_WORKSPACE
    assert back(ref(cfg), ref(qk_args()), ref(pair()), ref(pair()), P, P, P + 4, None) == lq.LQ_ERR_WORKSPACE
    assert back(ref(cfg), ref(qk_args(weight_q=None)), ref(pair()), ref(pair()), P, None, P, None) == lq.LQ_ERR_INVALID_ARG
    assert back(ref(cfg), ref(qk_args()), None, ref(pair()), None, None, None, None) == lq.LQ_ERR_INVALID_ARG
    none = qk_config(heads_k=0)                        # a key weight may be there, its gradient may not
    assert back(ref(none), ref(qk_args()), ref(pair()), ref(pair()), P, P, P, None) == lq.LQ_ERR_INVALID_ARG
    assert L.lq_qk_norm_rotate(ref(cfg), ref(qk_args()), None, None) == lq.LQ_ERR_INVALID_ARG


def test_the_binding_refuses_host_tensors():
    v, g = torch.zeros(4, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 2)
    for call in (lambda: lq.gated_scan(v, g), lambda: lq.qk_norm_rotate(v, v),
                 lambda: lq.gated_scan_backward(v, v, g, checkpoints=None)):
        with pytest.raises(AssertionError, match="CUDA"):
            call()


def test_packed_structs_are_the_structs():
    """The binding packs its calls with formats of the structs' sizes."""
    import struct
    for pack, cls in ((lq._pack_scan_config, lq.ScanConfig), (lq._pack_scan_args, lq.ScanArgs),
                      (lq._pack_scan_grads, lq.ScanGrads), (lq._pack_qk_config, lq.QkNormConfig),
                      (lq._pack_qk_args, lq.QkNormArgs), (lq._pack_qk_pair, lq.QkPair)):
        f = pack.__self__
        assert f.size == ctypes.sizeof(cls)
        values = [i + 1 for i in range(len(struct.unpack(f.format, bytes(f.size))))]
        flat, got = [], cls.from_buffer_copy(pack(*values))
        for n, t in cls._fields_:
            x = getattr(got, n)
            flat += [getattr(x, m) for m, _ in t._fields_] if t is lq.Strides else [x]
        assert flat == values, cls


def test_structs_match_the_header():
    """Field names and order of the binding's structs are the header's."""
    import re
    with open(lq.HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    for name, struct in (("lq_strides", lq.Strides), ("lq_scan_config", lq.ScanConfig), ("lq_scan_args", lq.ScanArgs),
                         ("lq_scan_grads", lq.ScanGrads), ("lq_qk_norm_config", lq.QkNormConfig),
                         ("lq_qk_norm_args", lq.QkNormArgs), ("lq_qk_pair", lq.QkPair)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        fields = [f.strip(" *") for line in body.split(";") if line.strip()
                  for f in re.sub(r"^\s*(const )?\w+\s", "", line.strip()).split(",")]
        assert fields == [n for n, _ in struct._fields_], name


def state_with_norm(batch=2, heads=4, d=64, **how):
    """A state's fields without its memory: what its calls check before anything reaches a device."""
    st = object.__new__(lq.DecodeState)
    st.__dict__.update(batch=batch, heads=heads, d=d, in_dtype=torch.bfloat16, qk_norm=how, _h=None,
                       device=torch.device("cpu"))
    return st


@pytest.mark.parametrize("q,k", [((2, 4, 64), (2, 1, 64)), ((2, 4, 64), (2, 4, 32)), ((2, 1, 64), (2, 4, 64)),
                                 ((1, 4, 64), (1, 4, 64)), ((2, 4, 64), None), ((2, 8, 32), (2, 8, 32))])
def test_a_state_refuses_queries_and_keys_of_other_heads(q, k):
    """The norm takes fewer key heads than query heads; the decode kernels read a key a head."""
    q, k = (None if s is None else torch.zeros(s, dtype=torch.bfloat16) for s in (q, k))
    v, g = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4)
    up = lambda x: None if x is None else torch.stack([x] * 3)  # noqa: E731
    mask = torch.ones(2, dtype=torch.uint8)
    st = state_with_norm()
    for call in (lambda: st.decode_step(q, k, v, g, g), lambda: st.prefill_tokens(up(q), up(k), up(v), up(g), up(g)),
                 lambda: st.prefill_sequences_tokens(up(q), up(k), up(v), up(g), up(g), mask)):
        with pytest.raises(AssertionError, match="batch, heads, d"):
            call()


@pytest.fixture
def host_tensors_pass(monkeypatch):
    """The binding's checks on host tensors, up to the library call (which the test sees refused or made)."""
    monkeypatch.setattr(lq, "_on", lambda x, stream: None)
    monkeypatch.setattr(lq, "_raw_stream", lambda device: 0)

    class Library:
        calls = []

        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return lambda *a: 64
            return lambda *a: self.calls.append(name) or lq.LQ_OK

    fake = Library()
    fake.calls.clear()
    monkeypatch.setattr(lq, "lib", lambda: fake)
    return fake.calls


def test_positions_and_frequencies_go_together(host_tensors_pass):
    q, pos = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    freq = torch.ones(16, dtype=torch.float64)
    for how in ({"positions": pos}, {"inv_freq": freq}, {"positions": pos, "inv_freq": freq[:0]}):
        for call in (lambda: lq.qk_norm_rotate(q, q, **how), lambda: lq.qk_norm_rotate_backward(q, q, q, q, **how)):
            with pytest.raises(AssertionError, match="positions and inv_freq"):
                call()
    st = state_with_norm(batch=3, heads=2)
    with pytest.raises(AssertionError, match="positions and inv_freq"):
        st.decode_step(q, q, q, q[..., 0], q[..., 0], positions=pos)
    assert host_tensors_pass == []
    lq.qk_norm_rotate(q, q, positions=pos, inv_freq=freq)
    lq.qk_norm_rotate(q, q)
    assert host_tensors_pass == ["lq_qk_norm_rotate"] * 2


def test_tensors_that_autograd_follows_are_refused(host_tensors_pass):
    """The results have no graph, so a loss on them would leave the leaves without a gradient."""
    leaf = lambda *s: torch.zeros(*s, requires_grad=True)  # noqa: E731
    q, w, g, h, m = torch.zeros(3, 2, 4, 64), torch.zeros(64), torch.zeros(3, 2, 4), torch.zeros(2, 4, 64), torch.zeros(99)
    ql, wl, gl, hl = leaf(3, 2, 4, 64), leaf(64), leaf(3, 2, 4), leaf(2, 4, 64)
    calls = [lambda: lq.gated_scan(ql, g), lambda: lq.gated_scan(q, gl), lambda: lq.gated_scan(q, g, gl),
             lambda: lq.gated_scan(q, g, g, hl), lambda: lq.gated_scan_backward(ql, q, g, checkpoints=m),
             lambda: lq.gated_scan_backward(q, ql, g, checkpoints=m), lambda: lq.qk_norm_rotate(ql, q),
             lambda: lq.qk_norm_rotate(q, ql), lambda: lq.qk_norm_rotate(q, q, weight_q=w, weight_k=wl),
             lambda: lq.qk_norm_rotate_backward(q, q, q, ql), lambda: lq.qk_norm_rotate_backward(q, ql, q, q)]
    for call in calls:
        with pytest.raises(AssertionError, match="requires a gradient"):
            call()
    assert host_tensors_pass == []
    with torch.no_grad():
        for call in calls:
            call()
    assert len(host_tensors_pass) == len(calls)
    st = state_with_norm(batch=2, heads=4, weight_q=wl)       # a state's calls have no gradients either way
    assert all(not x.requires_grad for x in st._normed(ql[0], q[0], None, None))


@pytest.mark.parametrize("strides", [(2, 0, 0, 1), (1, 0, 0, 1), (8, 16, 4, 1), (24, 120, 8, 1)])
def test_inputs_whose_tokens_overlap_are_taken(host_tensors_pass, strides):
    """Sliding windows over a sequence are views with contiguous channels like any other."""
    v = torch.zeros(1000).as_strided((5, 2, 3, 8), strides)
    out, _ = lq.gated_scan(v, v)
    gv, gg, _, _ = lq.gated_scan_backward(v, v, v, checkpoints=v.new_empty(64))
    for x in (out, gv, gg):
        assert x.shape == v.shape and x.stride(3) == 1 and len({x[i].data_ptr() for i in range(5)}) == 5
    if strides == (24, 120, 8, 1):                       # what is dense keeps its order
        assert out.stride() == gv.stride() == v.stride()
