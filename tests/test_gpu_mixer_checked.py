"""Convolution, scan and norms in the bounds-checked build: every form runs with a status of 0 and gives the
bits of the normal build."""
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn
from chunked_gated_delta_06_gb300 import binding, build

import test_gpu_conv as conv
import test_gpu_norm as norm
import test_gpu_scan as scan

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def checked():
    return build.build(checked=True)


def _same(checked, run):
    """run(status): tensors, the same through both builds."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = run(status)
    with binding.use_library(checked):
        got = run(status)
        torch.cuda.synchronize()
    assert int(status) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("lens, C, W, dtype, wider", [([70, 0, 1, 300], 1032, 4, BF, 8), ([5, 40], 7, 3, F32, 1),
                                                      ([200], 600, 2, F32, 0), ([33] * 9, 260, 4, BF, 3)])
def test_convolution(checked, lens, C, W, dtype, wider):
    c = conv.Case(lens, C, W, dtype, wider=wider)
    pool = torch.randn(len(lens) + 2, C, W - 1, device="cuda").to(dtype)
    idx = torch.arange(len(lens), 0, -1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(status):
        p, s = pool.clone(), pool.clone()
        y = gdn.short_conv_prefill_paged(c.x, c.w, c.cu, c.cu_dev, p, idx, device_status=slots, problem_status=status, **c.kw())
        z = gdn.short_conv_step(c.x[:len(lens)], c.w, s, idx, device_status=slots, **c.kw())
        return [*c.fwd(device_status=status), *c.bwd(device_status=status).values(), y, p, z, s]
    _same(checked, run)
    assert int(slots) == 0


@pytest.mark.parametrize("lens, C, Ns, G, dtype, wider, seg", [([70, 0, 1, 300], 264, 16, 1, BF, 16, 64), ([5, 40], 7, 8, 7, F32, 1, -1),
                                                               ([200], 130, 32, 2, F32, 0, 96), ([33] * 9, 300, 16, 3, BF, 3, 32),
                                                               ([90, 35], 520, 8, 1, BF, 0, 32)])
def test_scan(checked, lens, C, Ns, G, dtype, wider, seg):
    c = scan.Case(lens, C, Ns, G, dtype, wider=wider)
    N = len(lens)
    pool = torch.randn(N + 2, C, Ns, device="cuda")
    idx = torch.arange(N, 0, -1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(status):
        p, s = pool.clone(), pool.clone()
        y = gdn.selective_scan_prefill_paged(*c.args(), c.cu, c.cu_dev, p, idx, device_status=slots, problem_status=status,
                                             segment_tokens=seg, **c.kw())
        z = gdn.selective_scan_step(c.x[:N], c.dt[:N], c.A_log, c.B[:N], c.C[:N], s, idx, D=c.D, z=c.z[:N], dt_bias=c.bias,
                                    device_status=slots)
        kw = dict(device_status=status, segment_tokens=seg)
        return [*c.fwd(**kw), *c.bwd(**kw).values(), y, p, z, s]
    _same(checked, run)
    assert int(slots) == 0


@pytest.mark.parametrize("rows, D, dtype, residual", [(700, 128, BF, None), (9, 129, F32, F32), (5, 4096, BF, F32), (40, 264, BF, BF),
                                                      (3, 8192, F32, F32), (3, 8191, BF, BF)])
def test_norm(checked, rows, D, dtype, residual):
    c = norm.Case(rows, D, dtype, gate="silu", residual=residual, scale=residual is not None)

    def run(status):
        y, h = c.fwd()
        got = c.bwd(c.x if h is None else h)
        return [y, *(t for t in (h, *got.values()) if t is not None)]
    _same(checked, run)
