"""A wait of the gated scan that runs out leaves NaN in what came too late and in
all that depends on it, and nothing else.  gpu_scan_late_probe.cu compiles the
scan's own source with a wait that answers "not in time" at one step."""
import ctypes
import os
import subprocess

import pytest
import torch

from recurrent_state_quantization_lq_b200 import lq

pytestmark = pytest.mark.gpu
DEV = "cuda"
HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
BF, F32 = torch.bfloat16, torch.float32
ref = ctypes.byref


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("scanlate") / "libscanlate.so")
    subprocess.run(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "--expt-relaxed-constexpr",
                    "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "recurrent_state_quantization_lq_b200", "csrc"),
                    os.path.join(HERE, "gpu_scan_late_probe.cu"), "-o", out], check=True, capture_output=True, timeout=600)
    lib = ctypes.CDLL(out)
    lib.lq_test_scan_late.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int] * 2
    lib.lq_test_scan_late.restype = ctypes.c_int
    return lib


def s3(x):
    return tuple(x.stride()[:3])


@pytest.mark.parametrize("T,B,H,late_block", [(5000, 1, 2, 0), (700, 32, 16, 3)])
@pytest.mark.parametrize("dtype,chan", [(BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("step", [0, 1, 2])
def test_late_tokens_leave_nan_and_only_what_depends_on_them(probe, T, B, H, late_block, dtype, chan, step):
    """Few units run over clusters (the late CTA is a unit's first), many with a CTA each."""
    d = 128
    gen = torch.Generator().manual_seed(T)
    v, dy = (torch.randn(T, B, H, d, generator=gen).to(dtype).to(DEV) for _ in range(2))
    g = -0.1 * torch.rand(T, B, H, *([d] if chan else []), generator=gen).to(DEV)
    h0, dh = (torch.randn(B, H, d, generator=gen).to(DEV) for _ in range(2))
    marks = lq.gated_scan_checkpoints(v, g)
    out, last = lq.gated_scan(v, g, None, h0, checkpoints=marks)
    good = lq.gated_scan_backward(dy, v, g, checkpoints=marks, grad_last=dh)
    torch.cuda.synchronize()
    cfg = lq.ScanConfig(B, H, d, int(chan), int(dtype is BF), int(dtype is BF))
    args = lq.ScanArgs(n_tokens=T, v=v.data_ptr(), g=g.data_ptr(), h0=h0.data_ptr(), v_stride=s3(v), g_stride=s3(g))

    def units(x):                              # [unit][token][...], as one row a token
        return x.reshape(T, B * H, -1).transpose(0, 1)

    def split_point(x, want, late_first):
        """The token where NaN begins (ends): on one side all is NaN, on the other all as it should be."""
        x, want = units(x), units(want)
        others = [u for u in range(B * H) if u != unit]
        assert torch.equal(x[others], want[others])
        nan = x[unit].isnan()
        n = int(nan.any(-1).sum())
        cut = T - n if late_first else n
        lost, kept = (slice(cut, T), slice(0, cut)) if late_first else (slice(0, cut), slice(cut, T))
        assert nan[lost].all() and torch.equal(x[unit][kept], want[unit][kept])
        return cut

    unit = late_block                          # (block 0 is unit 0's first CTA, whatever the cluster's size)
    o, hl = torch.empty_like(out), torch.empty_like(last)
    args.out, args.h_last, args.out_stride = o.data_ptr(), hl.data_ptr(), s3(o)
    assert probe.lq_test_scan_late(ref(cfg), ref(args), None, late_block, -1) == 0
    assert torch.equal(o, out) and torch.equal(hl, last)
    assert probe.lq_test_scan_late(ref(cfg), ref(args), None, late_block, step) == 0
    cut = split_point(o, out, True)
    rows = 16 * (6 if chan else 7) // 8        # of 16 lanes
    chunk = rows * ((3 if dtype is BF else 2) if chan else (8 if dtype is BF else 4))
    assert cut in [step * r * chunk for r in range(1, 9)] and cut < T
    hl, want = hl.view(B * H, d), last.view(B * H, d)
    assert hl[unit].isnan().all() and torch.equal(hl[:unit], want[:unit]) and torch.equal(hl[unit + 1:], want[unit + 1:])

    args.out = args.h_last = None
    args.checkpoints = marks.data_ptr()
    gv, gg, gh = torch.empty_like(v), torch.empty_like(g), torch.empty_like(h0)
    grads = lq.ScanGrads(grad_out=dy.data_ptr(), grad_last=dh.data_ptr(), grad_v=gv.data_ptr(), grad_g=gg.data_ptr(),
                         grad_h0=gh.data_ptr(), grad_out_stride=s3(dy), grad_v_stride=s3(gv), grad_g_stride=s3(gg))
    assert probe.lq_test_scan_late(ref(cfg), ref(args), ref(grads), late_block, -1) == 0
    assert torch.equal(gv, good[0]) and torch.equal(gg, good[1]) and torch.equal(gh, good[3])
    assert probe.lq_test_scan_late(ref(cfg), ref(args), ref(grads), late_block, step) == 0
    cut = split_point(gv, good[0], False)
    assert split_point(gg, good[1], False) == cut and 0 < cut <= T
    chunk = 12 * (4 if dtype is BF and not chan else 2)
    assert cut % chunk == 0 or (cut == T and step == 0)
    gh, want = gh.view(B * H, d), good[3].view(B * H, d)
    assert gh[unit].isnan().all() and torch.equal(gh[:unit], want[:unit]) and torch.equal(gh[unit + 1:], want[unit + 1:])
