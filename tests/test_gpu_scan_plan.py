"""Scans that the library's own plan splits (tests/test_mixer_limits.py has that it does), several sequences and blocks
of channels, element by element against the 64-bit definition."""
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

from test_gpu_scan import GRADS, Case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens, C, Ns, G", [([300, 0, 150], 96, 16, 1), ([500, 260], 160, 8, 1), ([700, 33], 96, 32, 1)])
def test_split_by_the_plan(lens, C, Ns, G, dtype):
    for rate in (0.0, -4.0):   # (slow decays too, so that the states pass through the segments)
        c = Case(lens, C, Ns, G, dtype, seed=C, rate=rate)
        want = c.reference(grads=True)
        y, ht = c.fwd()
        c.check(dict(y=y, ht=ht), want, ("y", "ht"))
        c.check(c.bwd(), want, GRADS)
        pool = torch.cat([torch.zeros_like(c.h0[:1]), c.h0])
        idx = torch.arange(1, len(lens) + 1, dtype=torch.int32, device="cuda")
        yp = gdn.selective_scan_prefill_paged(*c.args(), c.cu, c.cu_dev, pool, idx, **c.kw())
        assert torch.equal(yp, y) and torch.equal(pool[1:], ht)
