"""Calls of the scan that the C header allows and the binding does not make."""
import ctypes

import pytest
import torch

import plain_ops
from recurrent_state_quantization_lq_b200 import lq

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {torch.float32: 0, torch.bfloat16: 1}
ref = ctypes.byref


def strides(x):
    return tuple(x.stride()[:3])


@pytest.mark.parametrize("d", [4, 12, 20, 100, 128, 252, 7])
@pytest.mark.parametrize("chan", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_a_gradient_of_the_state_alone_with_mixed_types(d, chan, dtype, out_dtype):
    """grad_out NULL with every pair of types: rows of out that are no whole pieces of 16 bytes (100 BF16
    channels: 200 bytes) stand for nothing then.  Token counts that leave rows of the last step empty."""
    for T in (1, 5, 333):
        B, H = 2, 3
        gen = torch.Generator().manual_seed(T + d)
        v = torch.randn(T, B, H, d, generator=gen).to(dtype).to(DEV)
        g = -0.1 * torch.rand(T, B, H, *([d] if chan else []), generator=gen).to(DEV)
        beta = torch.rand(T, B, H, generator=gen).to(DEV)
        h0, dh = (torch.randn(B, H, d, generator=gen).to(DEV) for _ in range(2))
        marks = lq.gated_scan_checkpoints(v, g)
        lq.gated_scan(v, g, beta, h0, checkpoints=marks, out_dtype=out_dtype)
        got = {"grad_v": torch.empty_like(v), "grad_g": torch.empty_like(g), "grad_beta": torch.empty_like(beta),
               "grad_h0": torch.empty_like(h0)}
        cfg = lq.ScanConfig(B, H, d, int(chan), TYPES[dtype], TYPES[out_dtype])
        args = lq.ScanArgs(n_tokens=T, v=v.data_ptr(), g=g.data_ptr(), beta=beta.data_ptr(),
                           checkpoints=marks.data_ptr(), v_stride=strides(v), g_stride=strides(g),
                           beta_stride=strides(beta))
        grads = lq.ScanGrads(grad_last=dh.data_ptr(), **{n: x.data_ptr() for n, x in got.items()},
                             grad_v_stride=strides(v), grad_g_stride=strides(g), grad_beta_stride=strides(beta))
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert lq.lib().lq_gated_scan_backward(ref(cfg), ref(args), ref(grads), stream) == lq.LQ_OK, lq.last_error()
        want = plain_ops.scan(v, g, beta, h0, None, None, dh)
        for n, x in got.items():
            plain_ops.check(x, want[n], x.dtype, (n, T))
