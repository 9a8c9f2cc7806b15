"""Decay-only linear attention and rotary positions in the bounds-checked build: every form runs
with a status of 0 and gives the bits of the normal build."""
import os
import re

import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn
from chunked_gated_delta_06_gb300 import binding, build

from test_gpu_linear import Case


def test_every_kernel_checks_its_accesses():
    # (in the source: an access outside is not made on purpose on any GPU)
    for name in ("gdn_linear.cu", "gdn_linear_tc.cu", "gdn_rope.cu"):
        text = open(os.path.join(build.CSRC, name)).read()
        for start in re.finditer(r"__global__", text):
            end = text.index("\n}\n", start.start())
            body = text[start.start():end]
            kernel = re.search(r"\b(k_\w+)\(", body).group(1)
            assert "in_range(" in body or "scan<" in body, kernel
    text = open(os.path.join(build.CSRC, "gdn_linear_tc.cu")).read()
    body = text[text.index("void scan("):text.index("// The scans of a call")]
    # states, slots and segment records by one checked accessor
    assert not re.search(r"(ps\.s0|ps\.s1|a\.pool|ps\.seg_state) \+", body)


@pytest.fixture(scope="module")
def checked():
    return build.build(checked=True)


@pytest.mark.gpu
@pytest.mark.parametrize("lens, H, HV, seg", [([130, 1, 300], 2, 4, -1), ([700, 0, 129], 1, 1, 2), ([640], 1, 2, 1),
                                              ([385, 90], 1, 3, 2), ([5, 0, 40] * 50, 1, 2, 0)])
def test_scans(checked, lens, H, HV, seg):
    c = Case(lens, H, HV)
    status, slots = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    pool = torch.randn(len(lens) + 2, HV, 128, 128, device="cuda")
    idx = torch.arange(len(lens), 0, -1, dtype=torch.int32, device="cuda")

    def run(**kw):
        p = pool.clone()
        o = gdn.linear_attn_prefill_paged(c.q, c.k, c.v, c.g, c.cu, c.cu_dev, p, idx, scan_segment_chunks=seg,
                                          device_status=slots, problem_status=kw.get("device_status"))
        gr = c.bwd(scan_segment_chunks=seg, **kw)
        return [*c.fwd(scan_segment_chunks=seg, **kw), o, p, *(gr[n] for n in ("dq", "dk", "dv", "dh0"))]
    want = run()
    with binding.use_library(checked):
        got = run(device_status=status)
        torch.cuda.synchronize()
    assert int(status) == 0 and int(slots) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_step_and_rope(checked):
    B, H, HV = 5, 2, 4
    q, k, v = (torch.randn(B, h, 128, device="cuda").to(torch.bfloat16) for h in (H, H, HV))
    g = -torch.rand(HV, device="cuda")
    pool = torch.randn(B + 1, HV, 128, 128, device="cuda")
    idx = torch.tensor([5, 2, 0, 1, 4], dtype=torch.int32, device="cuda")
    pos = torch.arange(B, dtype=torch.int32, device="cuda") * 1000
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        p = pool.clone()
        o = gdn.linear_attn_step(q, k, v, g, p, idx, device_status=status)
        out = [o, p]
        for rot, layout in ((128, "half"), (36, "interleaved"), (2, "half")):
            out += gdn.rope(q, k, pos, gdn.rope_frequencies(rot), layout=layout)
        return out
    want = run()
    with binding.use_library(checked):
        got = run()
        torch.cuda.synchronize()
    assert int(status) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
