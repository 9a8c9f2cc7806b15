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


class _Wide:
    """What the calls look at of a dense CUDA tensor of any size."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.is_cuda, self.device = dtype, torch.Size(shape), True, 0

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


def test_sizes_past_32_bits_are_refused(monkeypatch):
    # (as an int32 argument of the library 2^32 + 8 is 8)
    mixer._ready()

    class Library:
        def __getattr__(self, name):
            raise AssertionError("%s is reached" % name)
    monkeypatch.setattr(gdn.binding, "_lib", Library())
    monkeypatch.setattr(mixer.linear, "_current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: _Wide(torch.bfloat16, 1))
    monkeypatch.setattr(torch, "empty_like", lambda t: t)
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    big = (1 << 32) + 8
    row, w = _Wide(bf, 1, big), _Wide(f32, big)
    A, B = _Wide(f32, 8, 8), _Wide(bf, big, 1, 8)
    x, idx = _Wide(bf, big, 8), _Wide(i32, big)
    few, one, cu = _Wide(bf, 4, 8), _Wide(i32, 4), (np.array([0, 4], np.int32), _Wide(i32, 2))
    pool, Bf = _Wide(bf, big, 8, 3), _Wide(bf, 4, 1, 8)
    for call in (lambda: gdn.rms_norm_fwd(row, w), lambda: gdn.rms_norm_bwd(row, w, row),
                 lambda: gdn.short_conv_step(x, _Wide(f32, 8, 4), _Wide(bf, 4, 8, 3), idx),
                 lambda: gdn.short_conv_step(few, _Wide(f32, 8, 4), pool, one),
                 lambda: gdn.short_conv_prefill_paged(few, _Wide(f32, 8, 4), *cu, pool, _Wide(i32, 1)),
                 lambda: gdn.short_conv_fwd(_Wide(bf, 4, big), _Wide(f32, big, 4), *cu),
                 lambda: gdn.selective_scan_step(x, x, A, B, B, _Wide(f32, 4, 8, 8), idx),
                 lambda: gdn.selective_scan_step(few, few, A, Bf, Bf, _Wide(f32, big, 8, 8), one),
                 lambda: gdn.selective_scan_prefill_paged(few, few, A, Bf, Bf, *cu, _Wide(f32, big, 8, 8), _Wide(i32, 1)),
                 lambda: gdn.selective_scan_fwd(_Wide(bf, 4, big), _Wide(bf, 4, big), _Wide(f32, big, 8), Bf, Bf, *cu)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_batches_of_other_sizes_are_refused(offsets):
    x, B = torch.randn(1, 10, 8), torch.ones(1, 10, 1, 8)
    two = lambda t: torch.cat([t, t])  # noqa: E731
    rest = dict(dt=x, A_log=torch.ones(8, 8), B=B, C=B, z=x)
    gdn.selective_scan(x, **rest)
    with pytest.raises(ValueError, match="B must be 1"):
        gdn.short_conv(two(x), torch.ones(8, 4))
    for name in ("dt", "B", "C", "z"):   # (only the first of the two was read)
        with pytest.raises(ValueError, match="B must be 1"):
            gdn.selective_scan(x, **{**rest, name: two(rest[name])})
        with pytest.raises(ValueError, match="B must be 1"):
            gdn.selective_scan(x, **{**rest, name: rest[name][0]})   # (without a batch, unlike x)


def test_offsets_of_the_chunked_rule_changed_before_the_backward(monkeypatch):
    # a loop that reuses its offset buffers: the backward has the forward's host copy, and a device copy that changed
    # in place is an error
    seen = []

    def forward(q, k, v, g, beta, host, dev, **kw):
        return v * 2.0, None, host

    def backward(host, q, k, v, g, beta, d_o, **kw):
        seen.append(host.tolist())
        return dict(dq=q * 0, dk=k * 0, dv=v * 0, dg=g * 0, dbeta=beta * 0, dh0=None)
    monkeypatch.setattr(gdn.autograd.binding, "chunk_fwd", forward)
    monkeypatch.setattr(gdn.autograd.binding, "chunk_bwd", backward)
    q, g = torch.zeros(10, 1, 128, requires_grad=True), torch.zeros(10, 1)
    host, dev = torch.tensor([0, 3, 10], dtype=torch.int32), torch.tensor([0, 3, 10], dtype=torch.int32)
    o, _ = gdn.chunk_gated_delta_rule(q, q, q, g, g, cu_seqlens=dev, cu_seqlens_cpu=host)
    host[1] = 5
    o.sum().backward()
    assert seen == [[0, 3, 10]]
    o, _ = gdn.chunk_gated_delta_rule(q, q, q, g, g, cu_seqlens=dev, cu_seqlens_cpu=host)
    dev[1] = 5
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


def test_batches_of_other_sizes_are_refused_by_the_attentions(monkeypatch):
    monkeypatch.setattr(gdn.autograd.binding, "chunk_fwd", lambda q, k, v, *a, **kw: (v * 1.0, None, None))
    monkeypatch.setattr(gdn.autograd.linear, "linear_attn_fwd", lambda q, k, v, *a, **kw: (v * 1.0, None))
    q, g = torch.zeros(1, 10, 1, 128), torch.zeros(1, 10, 1)
    rule, linear = dict(q=q, k=q, v=q, g=g, beta=g), dict(q=q, k=q, v=q, log_decay=torch.zeros(1))
    for call, args in ((gdn.chunk_gated_delta_rule, rule), (gdn.linear_attention, linear)):
        assert call(**args)[0].shape == q.shape
        for name in ("q", "k", "v", "g", "beta") if call is gdn.chunk_gated_delta_rule else ("q", "k", "v"):
            with pytest.raises(ValueError, match="B must be 1"):
                call(**{**args, name: torch.cat([args[name]] * 2)})
            if name != "q":   # (a tensor without a batch lost all its tokens but the first)
                with pytest.raises(ValueError, match="B must be 1"):
                    call(**{**args, name: args[name][0]})
