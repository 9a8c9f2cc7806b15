"""The norms at the ends of their inputs' ranges: closed gates against the 64-bit definition, rows past fp32."""
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import mixer_reference as ref

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
