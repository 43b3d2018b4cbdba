"""Thin Python binding of liblq (include/lq.h): argument marshalling only.

Every step of the decode path runs in liblq's CUDA kernels; PyTorch supplies
device memory (the workspace and the input/output tensors) and streams.  If
liblq.so has not been built, importing the library raises: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# LQ_LIBRARY may name another build of the same C ABI, e.g. the bounds-checked
# liblq_checked.so (python -m recurrent_state_quantization_lq_b200.build --bounds-check)
LIB_PATH = os.environ.get("LQ_LIBRARY") or os.path.join(_HERE, "liblq.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "lq.h")

# enums of include/lq.h
LQ_OK, LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED, LQ_ERR_WORKSPACE, LQ_ERR_WINDOW_FULL = 0, 1, 2, 3, 4
LQ_ERR_RANGE, LQ_ERR_CUDA, LQ_ERR_DEVICE, LQ_ERR_STATE = 5, 6, 7, 8
GATE = {"scalar": 0, "gdn": 0, "channel": 1, "kda": 1}
MODE = {"window": 0, "naive": 1, "fp32": 2}
SELECT = {"l2": 0, "maxabs": 1}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
NORM = {"l2": 0, "rms": 1}
PAIRS = {"half": 0, "neighbours": 1}
ABSENT = ctypes.c_size_t(-1).value

LQ_DEVERR_BOUNDS = 4   # device error code: an index out of range (checked build; unit tickets in every build)

STATUS_NAMES = {0: "LQ_OK", 1: "LQ_ERR_INVALID_ARG", 2: "LQ_ERR_UNSUPPORTED", 3: "LQ_ERR_WORKSPACE",
                4: "LQ_ERR_WINDOW_FULL", 5: "LQ_ERR_RANGE", 6: "LQ_ERR_CUDA", 7: "LQ_ERR_DEVICE",
                8: "LQ_ERR_STATE"}


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "heads", "d_k", "d_v", "window", "n_comp_rows", "n_comp_cols", "gate", "mode",
        "smooth", "select", "in_dtype", "ragged")]


class Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "total_bytes", "err", "codes", "row_scale", "col_smooth", "comp_index", "comp_row_vec",
        "comp_col_vec", "gate_sum", "buf_delta", "buf_key", "buf_gate", "state_f32")] + \
        [("comp_index_stride", ctypes.c_int32), ("window_pad", ctypes.c_int32), ("fill", ctypes.c_size_t)]


EXPORT_REGIONS = ("codes", "row_scale", "col_smooth", "comp_index", "comp_row_vec", "comp_col_vec", "buf_delta",
                  "buf_key", "buf_gate", "gate_sum", "fill", "state_f32")


class Export(ctypes.Structure):
    """lq_export: destination pointers of lq_state_export (NULL = not copied)."""
    _fields_ = [(n, ctypes.c_void_p) for n in EXPORT_REGIONS]


class Strides(ctypes.Structure):
    """lq_strides, in elements."""
    _fields_ = [(n, ctypes.c_int64) for n in ("token", "seq", "head")]


class ScanConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "heads", "d", "gate", "in_dtype", "out_dtype")]


class ScanArgs(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("zero_past", ctypes.c_int32)] + \
        [(n, ctypes.c_void_p) for n in ("v", "g", "beta", "h0", "lengths", "out", "h_last", "checkpoints")] + \
        [(n, Strides) for n in ("v_stride", "g_stride", "beta_stride", "out_stride")]


class ScanGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("grad_out", "grad_last", "grad_v", "grad_g", "grad_beta", "grad_h0")] + \
        [(n, Strides) for n in ("grad_out_stride", "grad_v_stride", "grad_g_stride", "grad_beta_stride")]


class QkNormConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads_q", "heads_k", "d", "norm", "rot_dim", "pairs", "dtype")] + \
        [(n, ctypes.c_float) for n in ("eps", "q_scale")]


class QkNormArgs(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64)] + \
        [(n, ctypes.c_void_p) for n in ("q", "k", "positions", "inv_freq", "weight_q", "weight_k")] + \
        [(n, ctypes.c_int64) for n in ("q_token", "q_head", "k_token", "k_head")]


class QkPair(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p)] + \
        [(n, ctypes.c_int64) for n in ("q_token", "q_head", "k_token", "k_head")]


class LQError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}: {last_error()}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load liblq.so (built in-tree by ``python -m recurrent_state_quantization_lq_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m recurrent_state_quantization_lq_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32 = ctypes.c_void_p, ctypes.c_int32
        L.lq_workspace_bytes.argtypes = [ctypes.POINTER(Config)]
        L.lq_workspace_bytes.restype = ctypes.c_size_t
        L.lq_workspace_layout.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Layout)]
        L.lq_workspace_layout.restype = i32
        L.lq_state_create.argtypes = [ctypes.POINTER(Config), vp, ctypes.c_size_t, ctypes.POINTER(vp)]
        L.lq_state_create.restype = i32
        L.lq_prefill_state.argtypes = [vp, vp, vp]
        L.lq_prefill_state.restype = i32
        L.lq_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
        L.lq_decode_step.restype = i32
        L.lq_decode_step_active.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.lq_decode_step_active.restype = i32
        L.lq_window_flush.argtypes = [vp, vp]
        L.lq_window_flush.restype = i32
        L.lq_window_flush_pending.argtypes = [vp, vp]
        L.lq_window_flush_pending.restype = i32
        L.lq_prefill_sequences.argtypes = [vp, vp, vp, vp]
        L.lq_prefill_sequences.restype = i32
        L.lq_prefill_tokens.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp]
        L.lq_prefill_tokens.restype = i32
        L.lq_prefill_sequences_tokens.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp]
        L.lq_prefill_sequences_tokens.restype = i32
        L.lq_state_resume.argtypes = [vp, i32]
        L.lq_state_resume.restype = i32
        L.lq_window_fill.argtypes = [vp]
        L.lq_window_fill.restype = i32
        L.lq_state_export.argtypes = [vp, ctypes.POINTER(Export), vp]
        L.lq_state_export.restype = i32
        L.lq_device_status.argtypes = [vp, vp]
        L.lq_device_status.restype = i32
        L.lq_state_destroy.argtypes = [vp]
        L.lq_state_destroy.restype = i32
        L.lq_gated_scan_checkpoint_bytes.argtypes = [vp, i32]
        L.lq_gated_scan_checkpoint_bytes.restype = ctypes.c_size_t
        L.lq_gated_scan.argtypes = [vp, vp, vp]
        L.lq_gated_scan.restype = i32
        L.lq_gated_scan_backward.argtypes = [vp, vp, vp, vp]
        L.lq_gated_scan_backward.restype = i32
        L.lq_qk_norm_rotate.argtypes = [vp, vp, vp, vp]
        L.lq_qk_norm_rotate.restype = i32
        L.lq_qk_norm_rotate_workspace_bytes.argtypes = [vp]
        L.lq_qk_norm_rotate_workspace_bytes.restype = ctypes.c_size_t
        L.lq_qk_norm_rotate_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
        L.lq_qk_norm_rotate_backward.restype = i32
        L.lq_last_error_string.argtypes = []
        L.lq_last_error_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def header_symbols() -> list[str]:
    """Names of the entry points include/lq.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"LQ_API\s+[\w\s\*]+?\b(lq_\w+)\s*\(", text)


def last_error() -> str:
    return lib().lq_last_error_string().decode()


def make_config(batch: int, heads: int, d: int, window: int = 64, n_comp_rows: int = 2,
                n_comp_cols: int = 2, gate: str = "scalar", mode: str = "window", smooth: int = 1,
                select: str = "l2", in_dtype: torch.dtype = torch.bfloat16, ragged: bool = False) -> Config:
    return Config(batch, heads, d, d, window, n_comp_rows, n_comp_cols, GATE[gate], MODE[mode],
                  smooth, SELECT[select], DTYPE[in_dtype], int(ragged))


def workspace_bytes(cfg: Config) -> int:
    return lib().lq_workspace_bytes(ctypes.byref(cfg))


def workspace_layout(cfg: Config) -> Layout:
    L = Layout()
    st = lib().lq_workspace_layout(ctypes.byref(cfg), ctypes.byref(L))
    if st != LQ_OK:
        raise LQError(st, "lq_workspace_layout")
    return L


def _stream_ptr(stream, device) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(None if t is None else t.data_ptr())


# ------------------------------------------------------- stateless operators
# The structs above as packed bytes (a call's own, so threads share nothing):
# filling a ctypes struct takes longer than a small kernel runs.
_pack_scan_config = struct.Struct("6i").pack
_pack_scan_args = struct.Struct("2i8P12q").pack
_pack_scan_grads = struct.Struct("6P12q").pack
_pack_qk_config = struct.Struct("7i2f").pack
_pack_qk_args = struct.Struct("q6P4q").pack
_pack_qk_pair = struct.Struct("2P4q").pack
_NO_STRIDES = (0, 0, 0)


def _on(x: torch.Tensor, stream):
    """None when `x`'s device and the given stream are the current ones; else
    the context that makes them so, for the launch and what it allocates."""
    assert x.is_cuda, "a CUDA tensor is needed"
    if stream is None:
        return None if x.get_device() == torch.cuda.current_device() else torch.cuda.device(x.device)
    assert stream.device == x.device, (stream.device, x.device)
    return torch.cuda.stream(stream)


def _outside_autograd(*tensors):
    """Refuse tensors that autograd would follow: the results have no graph,
    and the gradients are calls of their own."""
    if torch.is_grad_enabled():
        for x in tensors:
            assert x is None or not x.requires_grad, \
                "a tensor requires a gradient, which autograd would not get through this call: call it under " \
                "torch.no_grad() or in an autograd.Function, with the operator's backward call for the gradients"


# the current stream's handle without a Stream object where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _refuse(x: torch.Tensor, what: str, device: int, dtype, shape):
    raise AssertionError(f"{what}: {x.dtype} {tuple(x.shape)} with strides {x.stride()} on device {x.get_device()}; "
                         f"wanted {dtype} {tuple(shape)} on device {device}, contiguous (rows: their channels)")


def _packed(x: torch.Tensor | None, what: str, device: int, dtype, shape) -> int:
    """The address of a contiguous tensor argument (0: None)."""
    if x is None:
        return 0
    if x.dtype is not dtype or x.shape != shape or x.get_device() != device or not x.is_contiguous():
        _refuse(x, what, device, dtype, shape)
    return x.data_ptr()


def _rows(x: torch.Tensor | None, what: str, device: int, dtype, shape):
    """The address and strides of a [T, batch, heads(, d)] argument of any
    strides whose channels are contiguous."""
    if x is None:
        return 0, _NO_STRIDES
    s = x.stride()
    if x.dtype is not dtype or x.shape != shape or x.get_device() != device or (len(s) == 4 and s[3] != 1 != shape[3]):
        _refuse(x, what, device, dtype, shape)
    return x.data_ptr(), s[:3]


def _result_like(x: torch.Tensor, dtype=None, make=torch.empty_like) -> torch.Tensor:
    """A tensor for results like x, in x's order where that leaves the channels
    contiguous (views whose tokens overlap may have none)."""
    y = make(x, dtype=dtype)
    return y if x.dim() < 4 or y.stride(3) == 1 else make(x, dtype=dtype, memory_format=torch.contiguous_format)


def _scan_config(v: torch.Tensor, g: torch.Tensor, out_dtype) -> bytes:
    assert v.dim() == 4, "v is [T, batch, heads, d]"
    T, B, H, d = v.shape
    chan = g.dim() == 4
    assert g.shape == (v.shape if chan else (T, B, H)), "g is [T, batch, heads] or [T, batch, heads, d]"
    return _pack_scan_config(B, H, d, chan, DTYPE[v.dtype], DTYPE[out_dtype])


def gated_scan_checkpoints(v: torch.Tensor, g: torch.Tensor) -> torch.Tensor:
    """The buffer that gated_scan(checkpoints=) fills for gated_scan_backward()
    on inputs of these shapes."""
    n = lib().lq_gated_scan_checkpoint_bytes(_scan_config(v, g, v.dtype), v.shape[0])
    if n == 0 and v.shape[0] > 0:
        raise LQError(LQ_ERR_INVALID_ARG, "lq_gated_scan_checkpoint_bytes")
    return v.new_empty(n // 4, dtype=torch.float32)


def _scan_inputs(v, g, beta, lengths, checkpoints, cfg, device):
    """Addresses of v, g, beta, lengths and checkpoints, and the strides of the first three."""
    T, B, H, _ = v.shape
    pv, sv = _rows(v, "v", device, v.dtype, v.shape)
    pg, sg = _rows(g, "g", device, torch.float32, g.shape)
    pb, sb = _rows(beta, "beta", device, torch.float32, (T, B, H))
    pl = _packed(lengths, "lengths", device, torch.int32, (B,))
    if checkpoints is None:
        return pv, pg, pb, pl, 0, sv, sg, sb
    need = lib().lq_gated_scan_checkpoint_bytes(cfg, T) // 4
    assert checkpoints.numel() >= need, "checkpoints of another shape: see gated_scan_checkpoints()"
    pc = _packed(checkpoints, "checkpoints", device, torch.float32, checkpoints.shape)
    return pv, pg, pb, pl, pc, sv, sg, sb


def gated_scan(v, g, beta=None, h0=None, *, lengths=None, out=None, h_last=None, checkpoints=None, out_dtype=None,
               want_out: bool = True, stream=None):
    """The gated linear recurrence h_t = exp(g_t) h_{t-1} + beta_t v_t over
    vector states (lq_gated_scan): v [T, batch, heads, d] (BF16 or FP32, any
    strides with contiguous channels; transpose a [batch, T, ...] tensor), g
    FP32 [T, batch, heads] or [T, batch, heads, d] (its sum over consecutive
    tokens at most 80, as g <= 0 always has it), beta FP32 [T, batch, heads]
    (None: 1), h0 FP32 [batch, heads, d] (None: zero), lengths int32 [batch]
    on the device (None: T).  Returns (out, h_last): every h_t in out_dtype
    (default v's), zero past a sequence's length, and the FP32 state after its
    last token.  `out` and `h_last` may be given (rows of `out` past a length
    then stay as they are; h_last may be h0); want_out=False skips `out`.
    `checkpoints` (gated_scan_checkpoints()) is filled for the backward pass."""
    _outside_autograd(v, g, beta, h0)
    on = _on(v, stream)
    if on is not None:
        with on:
            return gated_scan(v, g, beta, h0, lengths=lengths, out=out, h_last=h_last, checkpoints=checkpoints,
                              out_dtype=out_dtype, want_out=want_out)
    device, states = v.get_device(), v.shape[1:]
    out_dtype = out.dtype if out is not None else out_dtype or v.dtype
    cfg = _scan_config(v, g, out_dtype)
    pv, pg, pb, pl, pc, sv, sg, sb = _scan_inputs(v, g, beta, lengths, checkpoints, cfg, device)
    zero_past = out is None
    if zero_past and want_out:
        out = _result_like(v, out_dtype)
    if h_last is None:
        h_last = v.new_empty(states, dtype=torch.float32)
    po, so = _rows(out, "out", device, out_dtype, v.shape)
    args = _pack_scan_args(v.shape[0], zero_past, pv, pg, pb, _packed(h0, "h0", device, torch.float32, states), pl, po,
                           _packed(h_last, "h_last", device, torch.float32, states), pc, *sv, *sg, *sb, *so)
    st = lib().lq_gated_scan(cfg, args, _raw_stream(device))
    if st != LQ_OK:
        raise LQError(st, "lq_gated_scan")
    return out, h_last


def gated_scan_backward(grad_out, v, g, beta=None, *, checkpoints, grad_last=None, lengths=None, grad_v=None,
                        grad_g=None, grad_beta=None, grad_h0=None, stream=None):
    """The gradients of gated_scan() (lq_gated_scan_backward): v, g, beta and
    lengths as in the forward call, `checkpoints` as it filled them, grad_out
    like out (None: zero), grad_last FP32 like h_last (None: zero).  Returns
    (grad_v, grad_g, grad_beta, grad_h0); grad_beta is None without beta.
    Tokens past a length get zero, or stay as they are in a tensor given for
    the result."""
    _outside_autograd(grad_out, grad_last, v, g, beta)
    on = _on(v, stream)
    if on is not None:
        with on:
            return gated_scan_backward(grad_out, v, g, beta, checkpoints=checkpoints, grad_last=grad_last,
                                       lengths=lengths, grad_v=grad_v, grad_g=grad_g, grad_beta=grad_beta,
                                       grad_h0=grad_h0)
    device, states = v.get_device(), v.shape[1:]
    out_dtype = v.dtype if grad_out is None else grad_out.dtype
    cfg = _scan_config(v, g, out_dtype)
    pv, pg, pb, pl, pc, sv, sg, sb = _scan_inputs(v, g, beta, lengths, checkpoints, cfg, device)
    # rows past a length: zeroed by the kernel, unless a given tensor is to keep its own
    zero_past = grad_v is None and grad_g is None and grad_beta is None
    make = torch.empty_like if zero_past or lengths is None else torch.zeros_like
    grad_v = _result_like(v, None, make) if grad_v is None else grad_v
    grad_g = _result_like(g, None, make) if grad_g is None else grad_g
    if beta is not None and grad_beta is None:
        grad_beta = _result_like(beta, None, make)
    if grad_h0 is None:
        grad_h0 = v.new_empty(states, dtype=torch.float32)
    py, sy = _rows(grad_out, "grad_out", device, out_dtype, v.shape)
    pgv, sgv = _rows(grad_v, "grad_v", device, v.dtype, v.shape)
    pgg, sgg = _rows(grad_g, "grad_g", device, torch.float32, g.shape)
    pgb, sgb = _rows(grad_beta, "grad_beta", device, torch.float32, v.shape[:3])
    args = _pack_scan_args(v.shape[0], zero_past, pv, pg, pb, 0, pl, 0, 0, pc, *sv, *sg, *sb, 0, 0, 0)
    grads = _pack_scan_grads(py, _packed(grad_last, "grad_last", device, torch.float32, states), pgv, pgg, pgb,
                             _packed(grad_h0, "grad_h0", device, torch.float32, states), *sy, *sgv, *sgg, *sgb)
    st = lib().lq_gated_scan_backward(cfg, args, grads, _raw_stream(device))
    if st != LQ_OK:
        raise LQError(st, "lq_gated_scan_backward")
    return grad_v, grad_g, grad_beta, grad_h0


def _heads_of(x: torch.Tensor | None, what: str, device: int, dtype, shape):
    """The address, token stride and head stride of a [..., heads, d] argument."""
    if x is None:
        return 0, 0, 0
    s = x.stride()
    if x.dtype is not dtype or x.shape != shape or x.get_device() != device or s[-1] != 1 != shape[-1]:
        _refuse(x, what, device, dtype, shape)
    if len(s) == 3:
        token = s[0]
    else:                                      # the tokens of several leading dimensions lie at one stride
        token, n = 0, 1
        for size, step in zip(reversed(shape[:-2]), reversed(s[:-2])):
            if size == 1:
                continue
            token = step if n == 1 else token
            assert step == token * n, f"{what}: its leading dimensions are not one run of tokens"
            n *= size
    # a dimension of one entry may have any stride: it is none
    return x.data_ptr(), token, s[-2] if shape[-2] > 1 else shape[-1]


def _qk_inputs(q, k, positions, inv_freq, weight_q, weight_k, norm, eps, pairs, q_scale):
    """The packed config and args of a call."""
    device, lead, d, dtype = q.get_device(), q.shape[:-2], q.shape[-1], q.dtype
    assert k is None or (k.shape[:-2] == lead and k.dim() >= 2 and k.shape[-1] == d), "k is [..., heads_k, d], as q"
    pq, tq, hq = _heads_of(q, "q", device, dtype, q.shape)
    pk, tk, hk = _heads_of(k, "k", device, dtype, None if k is None else k.shape)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    assert (rot == 0) == (positions is None), "a rotation needs positions and inv_freq, both or neither"
    cfg = _pack_qk_config(q.shape[-2], 0 if k is None else k.shape[-2], d, NORM[norm], rot, PAIRS[pairs], DTYPE[dtype],
                          eps, q_scale)
    args = _pack_qk_args(lead.numel(), pq, pk, _packed(positions, "positions", device, torch.int32, lead),
                         _packed(inv_freq, "inv_freq", device, torch.float64, (rot // 2,)),
                         _packed(weight_q, "weight_q", device, torch.float32, (d,)),
                         _packed(weight_k, "weight_k", device, torch.float32, (d,)), tq, hq, tk, hk)
    return cfg, args


def _qk_pair(q, k, like_q, like_k, what) -> bytes:
    assert (k is None) == (like_k is None), what
    device, dtype = like_q.get_device(), like_q.dtype
    pq, tq, hq = _heads_of(q, what, device, dtype, like_q.shape)
    pk, tk, hk = _heads_of(k, what, device, dtype, None if k is None else like_k.shape)
    return _pack_qk_pair(pq, pk, tq, hq, tk, hk)


def qk_norm_rotate(q, k=None, *, positions=None, inv_freq=None, weight_q=None, weight_k=None, norm: str = "l2",
                   eps: float = 1e-6, pairs: str = "half", q_scale: float = 1.0, q_out=None, k_out=None, stream=None):
    """Normalise every head of q [..., heads_q, d] and k [..., heads_k, d]
    (BF16 or FP32; views into a fused projection will do), then rotate its
    first 2 * len(inv_freq) channels by positions * inv_freq and multiply q by
    q_scale (lq_qk_norm_rotate).  norm: "l2" or "rms"; weights FP32 [d] (None:
    1); positions int32 [...] and inv_freq FP64 [rot_dim / 2] (both None: no
    rotation); pairs: "half" (i with i + rot_dim / 2) or "neighbours" (2 i
    with 2 i + 1).  Returns (q_out, k_out), new tensors unless given; they may
    be q and k themselves."""
    _outside_autograd(q, k, weight_q, weight_k)
    return _qk_norm_rotate(q, k, positions, inv_freq, weight_q, weight_k, norm, eps, pairs, q_scale, q_out, k_out, stream)


def _qk_norm_rotate(q, k, positions=None, inv_freq=None, weight_q=None, weight_k=None, norm="l2", eps=1e-6, pairs="half",
                    q_scale=1.0, q_out=None, k_out=None, stream=None):
    on = _on(q, stream)
    if on is not None:
        with on:
            return _qk_norm_rotate(q, k, positions, inv_freq, weight_q, weight_k, norm, eps, pairs, q_scale, q_out, k_out)
    cfg, args = _qk_inputs(q, k, positions, inv_freq, weight_q, weight_k, norm, eps, pairs, q_scale)
    if q_out is None:
        q_out = q.new_empty(q.shape)
    if k is not None and k_out is None:
        k_out = k.new_empty(k.shape)
    st = lib().lq_qk_norm_rotate(cfg, args, _qk_pair(q_out, k_out, q, k, "an output"), _raw_stream(q.get_device()))
    if st != LQ_OK:
        raise LQError(st, "lq_qk_norm_rotate")
    return q_out, k_out


def qk_norm_rotate_backward(grad_q_out, grad_k_out, q, k=None, *, positions=None, inv_freq=None, weight_q=None,
                            weight_k=None, norm: str = "l2", eps: float = 1e-6, pairs: str = "half",
                            q_scale: float = 1.0, grad_q=None, grad_k=None, stream=None):
    """The gradients of qk_norm_rotate() (lq_qk_norm_rotate_backward): q, k and
    the keywords as in the forward call, grad_q_out and grad_k_out those of
    its results.  Returns (grad_q, grad_k, grad_weight_q, grad_weight_k), the
    last two FP32 [d], None where there is no weight (or are no keys)."""
    _outside_autograd(grad_q_out, grad_k_out, q, k, weight_q, weight_k)
    on = _on(q, stream)
    if on is not None:
        with on:
            return qk_norm_rotate_backward(grad_q_out, grad_k_out, q, k, positions=positions, inv_freq=inv_freq,
                                           weight_q=weight_q, weight_k=weight_k, norm=norm, eps=eps, pairs=pairs,
                                           q_scale=q_scale, grad_q=grad_q, grad_k=grad_k)
    cfg, args = _qk_inputs(q, k, positions, inv_freq, weight_q, weight_k, norm, eps, pairs, q_scale)
    if grad_q is None:
        grad_q = q.new_empty(q.shape)
    if k is not None and grad_k is None:
        grad_k = k.new_empty(k.shape)
    gwq = None if weight_q is None else torch.empty_like(weight_q)
    gwk = None if weight_k is None or k is None else torch.empty_like(weight_k)
    work = None
    if gwq is not None or gwk is not None:
        n = lib().lq_qk_norm_rotate_workspace_bytes(cfg)
        if n == 0:
            raise LQError(LQ_ERR_INVALID_ARG, "lq_qk_norm_rotate_workspace_bytes")
        work = q.new_empty(n, dtype=torch.uint8)
    st = lib().lq_qk_norm_rotate_backward(cfg, args, _qk_pair(grad_q_out, grad_k_out, q, k, "a gradient of an output"),
                                          _qk_pair(grad_q, grad_k, q, k, "a gradient of an input"), _ptr(gwq), _ptr(gwk),
                                          _ptr(work), _raw_stream(q.get_device()))
    if st != LQ_OK:
        raise LQError(st, "lq_qk_norm_rotate_backward")
    return grad_q, grad_k, gwq, gwk


class DecodeState:
    """A batch of (sequence, head) recurrent states of one layer, held by liblq.

    The workspace is a torch uint8 tensor on ``device``; its regions can be
    viewed with :meth:`view`.  All calls enqueue on ``stream`` (default: the
    current stream) and return without synchronizing.

    ``qk_norm``: keywords of :func:`qk_norm_rotate` (norm, weights, inv_freq,
    q_scale, ...; {} for the plain L2 norm).  The decode and prefill calls then
    take q and k as a projection gives them (any strides that it takes) and
    normalise and rotate them first; with inv_freq they want ``positions``
    int32 [batch], or [T, batch] for a prompt.  The rows of sequences that are
    inactive or not masked are then read too, and never used.
    """

    def __init__(self, batch: int, heads: int, d: int, *, window: int = 64, n_comp_rows: int = 2,
                 n_comp_cols: int = 2, gate: str = "scalar", mode: str = "window", smooth: int = 1,
                 select: str = "l2", in_dtype: torch.dtype = torch.bfloat16, ragged: bool = False,
                 device=None, qk_norm: dict | None = None):
        self.qk_norm = qk_norm
        self.cfg = make_config(batch, heads, d, window, n_comp_rows, n_comp_cols, gate, mode, smooth,
                               select, in_dtype, ragged)
        self.ragged = bool(ragged)
        dev = torch.device(device) if device is not None else torch.device("cuda")
        if dev.index is None:
            dev = torch.device(dev.type, torch.cuda.current_device())
        self.device = dev
        nbytes = workspace_bytes(self.cfg)
        if nbytes == 0:
            raise LQError(LQ_ERR_INVALID_ARG, "lq_workspace_bytes")
        self.layout = workspace_layout(self.cfg)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        h = ctypes.c_void_p()
        st = lib().lq_state_create(ctypes.byref(self.cfg), _ptr(self.workspace), nbytes, ctypes.byref(h))
        if st != LQ_OK:
            raise LQError(st, "lq_state_create")
        self._h = h
        self.batch, self.heads, self.d = batch, heads, d
        self.in_dtype = in_dtype
        self.per_channel_gate = GATE[gate] == 1

    # ------------------------------------------------------------------ calls
    def _check(self, st: int, what: str) -> None:
        if st != LQ_OK:
            raise LQError(st, what)

    def prefill(self, S0: torch.Tensor | None = None, stream=None) -> None:
        if S0 is not None:
            assert S0.dtype == torch.float32 and S0.is_contiguous() and S0.device == self.device
            assert S0.numel() == self.batch * self.heads * self.d * self.d
        self._check(lib().lq_prefill_state(self._h, _ptr(S0), _stream_ptr(stream, self.device)),
                    "lq_prefill_state")

    def _normed(self, q, k, positions, stream, n_tokens: int = 1):
        """q and k as the C ABI takes them: through qk_norm where the state has one."""
        if self.qk_norm is None:
            assert positions is None, "positions without qk_norm"
            return q, k
        for x in (q, k):            # the norm takes any number of heads, the state its own
            assert x is not None and x.shape[-2:] == (self.heads, self.d) and \
                x.numel() == n_tokens * self.batch * self.heads * self.d, \
                f"q and k are [batch, heads, d], for a prompt [T, batch, heads, d]: {None if x is None else tuple(x.shape)}"
        return _qk_norm_rotate(q, k, positions, stream=stream, **self.qk_norm)     # (no state's call has gradients)

    def decode_step(self, q, k, v, g, beta, out: torch.Tensor | None = None, stream=None,
                    active: torch.Tensor | None = None, positions: torch.Tensor | None = None) -> torch.Tensor:
        """One token for every sequence; on a ragged state, for the sequences
        with active[b] != 0 (uint8 [batch] on the device; None = all)."""
        q, k = self._normed(q, k, positions, stream)
        if out is None:
            out = torch.empty(self.batch, self.heads, self.d, dtype=torch.float32, device=self.device)
        for t, dt in ((q, self.in_dtype), (k, self.in_dtype), (v, self.in_dtype), (g, torch.float32),
                      (beta, torch.float32), (out, torch.float32)):
            assert t.dtype == dt and t.is_contiguous() and t.device == self.device, (t.dtype, t.device)
        if active is not None:
            assert active.dtype == torch.uint8 and active.numel() == self.batch and active.device == self.device
            self._check(lib().lq_decode_step_active(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                                    _ptr(active), _ptr(out), _stream_ptr(stream, self.device)),
                        "lq_decode_step_active")
        else:
            self._check(lib().lq_decode_step(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(out),
                                             _stream_ptr(stream, self.device)), "lq_decode_step")
        return out

    def flush(self, stream=None) -> None:
        """End the window (ragged: of every unit whose window is full)."""
        self._check(lib().lq_window_flush(self._h, _stream_ptr(stream, self.device)), "lq_window_flush")

    def flush_pending(self, stream=None) -> None:
        """Ragged: end the window of every unit holding buffered tokens."""
        self._check(lib().lq_window_flush_pending(self._h, _stream_ptr(stream, self.device)),
                    "lq_window_flush_pending")

    def prefill_sequences(self, S0: torch.Tensor | None, mask: torch.Tensor, stream=None) -> None:
        """Ragged: restart the sequences with mask[b] != 0 (uint8 [batch] on the
        device) from S0 (FP32 [batch, heads, d, d]; None = zero state)."""
        if S0 is not None:
            assert S0.dtype == torch.float32 and S0.is_contiguous() and S0.device == self.device
            assert S0.numel() == self.batch * self.heads * self.d * self.d
        assert mask.dtype == torch.uint8 and mask.numel() == self.batch and mask.device == self.device
        self._check(lib().lq_prefill_sequences(self._h, _ptr(S0), _ptr(mask), _stream_ptr(stream, self.device)),
                    "lq_prefill_sequences")

    def prefill_tokens(self, q, k, v, g, beta, S0: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       stream=None, positions: torch.Tensor | None = None) -> torch.Tensor | None:
        """Run the FP32 recurrence over a prompt (inputs [T, batch, heads, ...]
        as for decode_step, stacked over tokens) from S0 (None = zero state) and
        encode its final state as the window-start state.  Writes the prompt's
        outputs into `out` ([T, batch, heads, d] FP32) when given."""
        q, k = self._normed(q, k, positions, stream, v.shape[0])
        T = q.shape[0]
        for t, dt in ((q, self.in_dtype), (k, self.in_dtype), (v, self.in_dtype), (g, torch.float32),
                      (beta, torch.float32)):
            assert t.dtype == dt and t.is_contiguous() and t.device == self.device and t.shape[0] == T, t.dtype
        if out is not None:
            assert out.dtype == torch.float32 and out.is_contiguous() and out.device == self.device
            assert out.numel() == T * self.batch * self.heads * self.d
        if S0 is not None:
            assert S0.dtype == torch.float32 and S0.is_contiguous() and S0.device == self.device
            assert S0.numel() == self.batch * self.heads * self.d * self.d
        self._check(lib().lq_prefill_tokens(self._h, _ptr(S0), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), T,
                                            _ptr(out), _stream_ptr(stream, self.device)), "lq_prefill_tokens")
        return out

    def prefill_sequences_tokens(self, q, k, v, g, beta, mask: torch.Tensor, lengths: torch.Tensor | None = None,
                                 S0: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                 stream=None, positions: torch.Tensor | None = None) -> torch.Tensor | None:
        """Ragged: restart the sequences with mask[b] != 0 from S0 (None = zero)
        through their prompts: inputs [T, batch, heads, ...] padded to T tokens,
        lengths int32 [batch] on the device (None = T for every sequence)."""
        q, k = self._normed(q, k, positions, stream, v.shape[0])
        T = q.shape[0]
        for t, dt in ((q, self.in_dtype), (k, self.in_dtype), (v, self.in_dtype), (g, torch.float32),
                      (beta, torch.float32)):
            assert t.dtype == dt and t.is_contiguous() and t.device == self.device and t.shape[0] == T, t.dtype
        assert mask.dtype == torch.uint8 and mask.numel() == self.batch and mask.device == self.device
        if lengths is not None:
            assert lengths.dtype == torch.int32 and lengths.numel() == self.batch and lengths.device == self.device
        if out is not None:
            assert out.dtype == torch.float32 and out.is_contiguous() and out.device == self.device
            assert out.numel() == T * self.batch * self.heads * self.d
        if S0 is not None:
            assert S0.dtype == torch.float32 and S0.is_contiguous() and S0.device == self.device
            assert S0.numel() == self.batch * self.heads * self.d * self.d
        self._check(lib().lq_prefill_sequences_tokens(self._h, _ptr(S0), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                                      _ptr(beta), T, _ptr(lengths), _ptr(mask), _ptr(out),
                                                      _stream_ptr(stream, self.device)),
                    "lq_prefill_sequences_tokens")
        return out

    def checkpoint(self, stream=None) -> tuple[torch.Tensor, int]:
        """A copy of the whole state: the workspace bytes and the shared-window
        count (0 on a ragged state, whose counts are in the workspace)."""
        status = self.device_status(stream)
        if status != LQ_OK:
            raise LQError(status, "checkpoint of a state with a device error")
        return self.workspace.clone(), max(self.fill, 0)

    def resume(self, workspace: torch.Tensor, n_buf: int) -> None:
        """Continue from a checkpoint() of a state with the same configuration."""
        assert workspace.dtype == torch.uint8 and workspace.numel() == self.workspace.numel()
        self.workspace.copy_(workspace)
        torch.cuda.synchronize(self.device)
        self._check(lib().lq_state_resume(self._h, int(n_buf)), "lq_state_resume")

    @property
    def fill(self) -> int:
        """Tokens buffered in the shared window; -1 on a ragged state (see fills())."""
        return lib().lq_window_fill(self._h)

    def fills(self) -> torch.Tensor:
        """Tokens buffered per (sequence, head) (read through lq_state_export,
        whatever the device error word holds)."""
        return self.export(["fill"], check=False)["fill"]

    def export_shapes(self) -> dict:
        """Dtype and packed shape of every region lq_state_export can copy for
        this state (regions the mode does not keep are absent)."""
        L, c = self.layout, self.cfg
        B, H, d, W = c.batch, c.heads, c.d_k, c.window
        key_dt = torch.float32 if (c.gate == 1 or c.in_dtype == 0) else torch.bfloat16
        spec = {
            "codes": (torch.int8, (B, H, d, d)),
            "row_scale": (torch.float32, (B, H, d)),
            "col_smooth": (torch.float32, (B, H, d)),
            "comp_index": (torch.int32, (B, H, c.n_comp_rows + c.n_comp_cols)),
            "comp_row_vec": (torch.float32, (B, H, c.n_comp_rows, d)),
            "comp_col_vec": (torch.float32, (B, H, c.n_comp_cols, d)),
            "buf_delta": (torch.float32, (B, H, W, d)),
            "buf_key": (key_dt, (B, H, W, d)),
            "buf_gate": (torch.float32, (B, H, W)),
            "gate_sum": (torch.float64, (B, H, d if c.gate == 1 else 1)),
            "fill": (torch.int32, (B, H)),
            "state_f32": (torch.float32, (B, H, d, d)),
        }
        present = {n for n in EXPORT_REGIONS if n != "fill" and getattr(L, n) != ABSENT}
        if c.mode == MODE["window"]:
            present.add("fill")
        return {n: spec[n] for n in EXPORT_REGIONS if n in present}

    def export(self, names=None, device="cpu", stream=None, check: bool = True) -> dict:
        """Copy state regions out through lq_state_export into new tensors on
        `device` (host tensors are pinned).  names: regions to copy (None = all
        this state keeps).  Synchronizes the stream.  Raises LQError when the
        device error word is set, unless check is False."""
        shapes = self.export_shapes()
        names = list(shapes) if names is None else list(names)
        dev = torch.device(device)
        pin = dev.type == "cpu" and torch.cuda.is_available()
        out, dst = {}, Export()
        for n in names:
            if n not in shapes:
                raise KeyError(f"this state keeps no {n}")
            dt, shape = shapes[n]
            x = torch.empty(shape, dtype=dt, device=dev, pin_memory=pin)
            out[n] = x
            if x.numel():
                setattr(dst, n, x.data_ptr())
        st = lib().lq_state_export(self._h, ctypes.byref(dst), _stream_ptr(stream, self.device))
        if st != LQ_OK and (check or st in (LQ_ERR_INVALID_ARG, LQ_ERR_STATE, LQ_ERR_CUDA)):
            raise LQError(st, "lq_state_export")
        return out

    def read(self, name: str, device="cpu", check: bool = True) -> torch.Tensor:
        """One region of the state, copied out through lq_state_export."""
        return self.export([name], device=device, check=check)[name]

    def device_status(self, stream=None) -> int:
        """Synchronize and return the status of the device error word (LQ_OK if clean)."""
        return lib().lq_device_status(self._h, _stream_ptr(stream, self.device))

    # ------------------------------------------------------------ inspection
    def view(self, name: str) -> torch.Tensor | None:
        """A writable tensor view of one workspace region, laid out as lq_layout
        says (internal layout: read the state with export(); this is for
        writing a state in, as a checkpoint restore does)."""
        L, c = self.layout, self.cfg
        off = getattr(L, name)
        if off == ABSENT:
            return None
        N, d = c.batch * c.heads, c.d_k
        gd = d if c.gate == 1 else 1
        key_dt = torch.float32 if (c.gate == 1 or c.in_dtype == 0) else torch.bfloat16
        nc = L.comp_index_stride
        spec = {
            "err": (torch.int32, (64,)),
            "codes": (torch.int8, (c.batch, c.heads, d, d)),
            "row_scale": (torch.float32, (c.batch, c.heads, d)),
            "col_smooth": (torch.float32, (c.batch, c.heads, d)),
            "comp_index": (torch.int32, (c.batch, c.heads, nc)),
            "comp_row_vec": (torch.float32, (c.batch, c.heads, c.n_comp_rows, d)),
            "comp_col_vec": (torch.float32, (c.batch, c.heads, c.n_comp_cols, d)),
            "gate_sum": (torch.float64, (c.batch, c.heads, gd)),
            "buf_delta": (torch.float32, (c.batch, c.heads, c.window, d)),
            "buf_key": (key_dt, (c.batch, c.heads, c.window, d)),
            "buf_gate": (torch.float32, (c.batch, c.heads, L.window_pad)),
            "state_f32": (torch.float32, (c.batch, c.heads, d, d)),
            "fill": (torch.int32, (c.batch, c.heads)),
        }[name]
        dt, shape = spec
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        return self.workspace[off:off + nbytes].view(dt).view(shape)

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().lq_state_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
