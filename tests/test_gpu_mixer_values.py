"""The convolution, the scan and the norms at the ends of their inputs' ranges: closed gates, tokens without a step and
far sums against the 64-bit definition, rows past fp32."""
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import mixer_reference as ref
import test_gpu_conv
import test_gpu_scan

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("D", [64, 129, 256, 1000, 4096, 8191])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_gates_that_are_closed(gate, dtype, D):
    # gates down to the type's lowest value, as a masked place has it: a closed gate's outputs and gradients are 0, below
    # 1e-30 from -80 on
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    rn = lambda *s, t=dtype: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    x, z, dy, w = rn(9, D), rn(9, D), rn(9, D), rn(D, t=F32)
    ends = [-80.0, -88.0, -89.0, -100.0, -1e4, -1e30, torch.finfo(dtype).min, 1e4]
    for i, end in enumerate(ends):
        z[i, i::7] = end
    z[8] = torch.finfo(dtype).min   # (a whole row)
    y, _ = gdn.rms_norm_fwd(x, w, z=z, gate=gate)
    want, off = ref.norm(x, w, z, gate)
    ref.check("y", y, want, off + ref.HALF[dtype] * want.abs() + 1e-30)
    got = gdn.rms_norm_bwd(x, w, dy, z=z, gate=gate)
    for name, (v, off) in ref.norm_bwd(x, w, dy, z, gate=gate).items():
        if got[name] is not None:
            ref.check(name, got[name], v, off + ref.HALF[got[name].dtype] * v.abs() + 1e-30)
    closed = z < -1e3
    assert closed.any() and not got["dz"][closed].any() and not got["dx"][8].any()


@pytest.mark.parametrize("D", [128, 129, 4096])
def test_rows_whose_squares_leave_fp32_are_zeros(D):
    x = torch.randn(5, D, device="cuda")
    x[2] = 1e25
    y, _ = gdn.rms_norm_fwd(x, torch.ones(D, device="cuda"))
    assert not y[2].any() and y[[0, 1, 3, 4]].abs().sum(1).gt(0).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("seg", [-1, 32])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scans_of_closed_gates_and_steps(dtype, seg):
    # a masked token has the type's lowest value as its step, its gate, or both
    low = torch.finfo(dtype).min
    c = test_gpu_scan.Case([70, 1, 33], 40, 16, 2, dtype, seed=5, rate=-2.0)
    c.dt[::5], c.z[::3] = low, low
    c.dt[3:9, ::2], c.z[1::7, 1::2] = -300.0, -1e30
    want = c.reference(grads=True)
    y, ht = c.fwd(segment_tokens=seg)
    c.check(dict(y=y, ht=ht), want, ("y", "ht"))
    got = c.bwd(segment_tokens=seg)
    c.check(got, want, test_gpu_scan.GRADS)
    assert not y[::3].any() and not got["dz"][::3].any() and not got["ddt"][::5].any()
    # one such token a row
    pool = torch.cat([torch.zeros_like(c.h0[:1]), c.h0])
    idx = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    one = [t[:3] if t.shape[0] == 104 else t for t in c.args()]
    y1 = gdn.selective_scan_step(*one, pool, idx, D=c.D, z=c.z[:3], dt_bias=c.bias)
    assert not y1[0].any() and torch.equal(pool[1], c.h0[0]) and torch.isfinite(y1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_convolutions_far_from_zero(dtype):
    c = test_gpu_conv.Case([70, 2, 33], 24, 4, dtype, seed=2)
    for i, far in enumerate([-80.0, -88.5, -1e4, -1e30, 1e4]):
        c.bias[i::9] = far
    c.check_fwd(*c.fwd())
    _, _, g, m = c.reference(grads=True)
    got = c.bwd()
    for name, key in (("dx", "dx"), ("dw", "dw"), ("dbias", "db"), ("dh0", "dh0")):
        ref.check(name, got[name], g[key], m[key] + ref.HALF[got[name].dtype] * g[key].abs() + 1e-30)
