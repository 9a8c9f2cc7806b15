"""The norm with its gate and residual on the GPU against its 64-bit definition: widths, types, gates,
scaled branches, gradients."""
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import mixer_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, rows, D, dtype=BF, gate=None, residual=None, scale=False, offset=0.0, eps=1e-6, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rn = lambda *s, t=dtype: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
        self.x, self.w = rn(rows, D), rn(D, t=F32)
        self.z = rn(rows, D) * 3 if gate else None
        self.residual = rn(rows, D, t=residual) if residual else None
        self.scale = rn(D, t=F32) if scale else None
        self.dy, self.dh = rn(rows, D), rn(rows, D, t=residual) if residual else None
        self.kw = dict(gate=gate or "silu", eps=eps, offset=offset)
        self.t = dtype

    def fwd(self):
        return gdn.rms_norm_fwd(self.x, self.w, z=self.z, residual=self.residual, scale=self.scale, **self.kw)

    def bwd(self, h, dh=True):
        return gdn.rms_norm_bwd(h, self.w, self.dy, z=self.z, dh=self.dh if dh else None, scale=self.scale,
                                x=None if self.scale is None else self.x, **self.kw)

    def check(self):
        y, h = self.fwd()
        assert (h is None) == (self.residual is None)
        at = self.x
        if h is not None:
            branch = self.x.double() * (1 if self.scale is None else self.scale.double())
            want = self.residual.double() + branch
            ref.check("h", h, want, ref.HALF[h.dtype] * want.abs() + 2.0 ** -23 * (branch.abs() + self.residual.abs()) + 1e-30)
            at = h
        kw = dict(self.kw, z=self.z)
        want, off = ref.norm(at, self.w, **kw)
        ref.check("y", y, want, off + ref.HALF[self.t] * want.abs() + 1e-30)
        got = self.bwd(at)
        want = ref.norm_bwd(at, self.w, self.dy, dh=self.dh, scale=self.scale, x=self.x, **kw)
        for name, value in got.items():
            there = name in want and (name != "dresidual" or self.residual is not None)
            assert (value is not None) == there, name
            if there:
                v, off = want[name]
                ref.check(name, value, v, off + ref.HALF[value.dtype] * v.abs() + 1e-30)


@pytest.mark.parametrize("rows, D", [(1, 1), (3, 3), (5, 8), (33, 128), (7, 96), (2, 129), (40, 256), (3, 1000), (5, 1024),
                                     (3, 2047), (4, 2048), (2, 4096), (3, 5120), (2, 8191), (2, 8192), (3000, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_and_gradient(rows, D, dtype):
    Case(rows, D, dtype).check()
    Case(rows, D, dtype, gate="silu", seed=1).check()
    Case(rows, D, dtype, gate="sigmoid", residual=F32, scale=True, offset=1.0, seed=2).check()
    Case(rows, D, dtype, residual=dtype, seed=3).check()


def test_the_stream_without_a_gradient_of_its_own():
    c = Case(9, 64, residual=F32)
    _, h = c.fwd()
    got = c.bwd(h, dh=False)
    want = ref.norm_bwd(h, c.w, c.dy, **c.kw)
    for n in ("dx", "dresidual"):
        v, off = want[n]
        ref.check(n, got[n], v, off + ref.HALF[got[n].dtype] * v.abs() + 1e-30)
    # one type, no scale: the branch's gradient is the stream's, one tensor
    c = Case(9, 64, residual=BF)
    got = c.bwd(c.fwd()[1])
    assert got["dx"] is got["dresidual"]


def test_rows_of_zeros_and_infinities_stay_their_own():
    c = Case(6, 128, gate="silu")
    c.x[1] = 0
    c.x[3, 5] = float("inf")
    y, _ = c.fwd()
    assert not y[1].any() and not torch.isfinite(y[3]).all()
    assert torch.isfinite(y[[0, 1, 2, 4, 5]]).all()
    c = Case(6, 128, eps=0.0)
    c.x[1] = 0
    y, _ = c.fwd()
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2, 3, 4, 5]]).all()   # 0 / 0


def test_no_rows():
    c = Case(0, 64, gate="silu")
    y, _ = c.fwd()
    assert y.shape == (0, 64)
    assert not c.bwd(c.x)["dweight"].any()


@pytest.mark.parametrize("residual, scale", [(None, False), (F32, True), (BF, False)])
def test_autograd_and_leading_dimensions(residual, scale):
    c = Case(24, 96, gate="silu", residual=residual, scale=scale)
    leaf = lambda t: None if t is None else t.detach().clone().view(2, 12, 96).requires_grad_()  # noqa: E731
    x, z, r = leaf(c.x), leaf(c.z), leaf(c.residual)
    w = c.w.clone().requires_grad_()
    s = None if c.scale is None else c.scale.clone().requires_grad_()
    out = gdn.rms_norm(x, w, z=z, residual=r, scale=s)
    y, h = out if residual else (out, None)
    dy = c.dy.view(2, 12, 96)
    torch.autograd.backward([y] if h is None else [y, h], [dy] if h is None else [dy, c.dh.view(2, 12, 96)])
    want = c.bwd(c.fwd()[1] if residual else c.x)
    for t, n in ((x, "dx"), (w, "dweight"), (z, "dz"), (r, "dresidual"), (s, "dscale")):
        if t is not None:
            assert torch.equal(t.grad.view(want[n].shape), want[n]), n
    if residual:   # the stream alone
        x2 = leaf(c.x)
        gdn.rms_norm(x2, c.w, residual=r.detach(), scale=s)[1].sum().backward()
        ones = torch.ones(96, device="cuda") if s is None else s.detach()
        assert torch.equal(x2.grad, ones.to(BF).expand(2, 12, 96))


def test_streams_and_graphs():
    c = Case(50, 128, gate="silu", residual=F32, scale=True)
    h = c.fwd()[1]
    want = c.bwd(h)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.bwd(h)
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = c.fwd()
        got = c.bwd(h)
    c.x.copy_(torch.randn_like(c.x))
    graph.replay()
    want_y, want_h = c.fwd()
    want = c.bwd(want_h)
    assert torch.equal(y, want_y) and all(torch.equal(got[n], want[n]) for n in want)
