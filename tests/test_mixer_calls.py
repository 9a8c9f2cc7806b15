"""The differentiable functions' handling of their arguments, with the kernels' calls replaced: nothing is launched."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn
from chunked_gated_delta_06_gb300 import mixer


@pytest.fixture
def offsets(monkeypatch):
    """The host and device offsets that the forward calls get."""
    seen = []

    def forward(x, *rest, **kw):
        host = next(i for i, a in enumerate(rest) if type(a) is np.ndarray)
        seen.append((rest[host], rest[host + 1]))
        return x * 2.0, None
    monkeypatch.setattr(mixer, "short_conv_fwd", forward)
    monkeypatch.setattr(mixer, "selective_scan_fwd", forward)
    return seen


def _mixers(**kw):
    x, B = torch.randn(10, 8), torch.ones(10, 1, 8)
    gdn.short_conv(x, torch.ones(8, 4), **kw)
    gdn.selective_scan(x, x, torch.ones(8, 8), B, B, **kw)


@pytest.mark.parametrize("make", [list, np.array, lambda v: np.array(v, np.int32), torch.tensor])
def test_offsets_of_the_host_alone(offsets, make):
    # the sequences are the caller's, not one of all tokens
    _mixers(cu_seqlens_cpu=make([0, 3, 3, 10]))
    _mixers(cu_seqlens=torch.tensor([0, 3, 3, 10]))
    assert len(offsets) == 4
    for host, dev in offsets:
        assert host.dtype == np.int32 and host.tolist() == [0, 3, 3, 10]
        assert dev.dtype == torch.int32 and dev.tolist() == [0, 3, 3, 10]


def test_no_offsets_are_one_sequence(offsets):
    _mixers()
    assert [(host.tolist(), dev.tolist()) for host, dev in offsets] == [([0, 10], [0, 10])] * 2


def test_offsets_of_the_host_alone_of_the_attentions(monkeypatch):
    # (the device's offsets were those of one sequence, shorter than the call reads them)
    seen = []

    def chunk(q, k, v, g, beta, host, dev, **kw):
        seen.append((host.tolist(), dev.tolist()))
        return v * 1.0, None, None

    def linear(q, k, v, log_decay, host, dev, **kw):
        seen.append((host.tolist(), dev.tolist()))
        return v * 1.0, None
    monkeypatch.setattr(gdn.autograd.binding, "chunk_fwd", chunk)
    monkeypatch.setattr(gdn.autograd.linear, "linear_attn_fwd", linear)
    q, g = torch.zeros(10, 1, 128), torch.zeros(10, 1)
    for kw in (dict(cu_seqlens_cpu=[0, 3, 10]), dict(cu_seqlens=torch.tensor([0, 3, 10])),
               dict(cu_seqlens=torch.tensor([0, 3, 10]), cu_seqlens_cpu=np.array([0, 3, 10])), {}):
        gdn.chunk_gated_delta_rule(q, q, q, g, g, **kw)
        gdn.linear_attention(q, q, q, torch.zeros(1), **kw)
    assert seen == [([0, 3, 10],) * 2] * 6 + [([0, 10],) * 2] * 2
