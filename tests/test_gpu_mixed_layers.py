"""The example layers: a training step, the same tokens served by prefill and steps, and the gradients of the
selective layer against 64 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import mixer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixed_layers.py")
    spec = importlib.util.spec_from_file_location("mixed_layers", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_served_tokens_match_the_packed_forward(example):
    # the two paths round alike but in the matrix products (their order) and the delta rule (bf16 states of
    # chunks): some ten values of 2^-8 at most on the way, a small multiple of it in the norm of all outputs
    torch.manual_seed(0)
    assert example.main() < 8 * 2.0 ** -8


def test_gradients_of_the_selective_layer(example):
    # convolution, scan and a residual norm in fp32 against the same chain in 64 bits, the gradients of
    # each taken by its formulas
    hidden, channels = 24, 40
    torch.manual_seed(1)
    layer = example.SelectiveLayer(hidden, channels, Ns=8, rank=8, dtype=torch.float32)
    cu = [0, 9, 9, 30]
    cu_host, cu_dev = np.array(cu, np.int32), torch.tensor(cu, dtype=torch.int32, device="cuda")
    u, stream = torch.randn(30, hidden, device="cuda"), torch.randn(30, hidden, device="cuda")
    norm, dy, dh = torch.randn(hidden, device="cuda"), torch.randn(30, hidden, device="cuda"), torch.randn(30, hidden, device="cuda")
    w = norm.clone().requires_grad_()
    s = stream.clone().requires_grad_()
    assert not torch.backends.cuda.matmul.allow_tf32   # (torch's default: fp32 products are fp32)
    y, h = gdn.rms_norm(layer.train(u, cu_dev, cu_host), w, residual=s)
    torch.autograd.backward([y, h], [dy, dh])

    # forward in 64 bits
    d = lambda t: t.detach().double()  # noqa: E731
    W_in, W_x, W_dt, W_out = (d(getattr(layer, n)) for n in ("w_in", "w_x", "w_dt", "w_out"))
    x0, z = (d(u) @ W_in).split([channels, channels], -1)
    (x, _), _, _, _ = ref.conv(x0, layer.conv.detach(), cu, layer.bias.detach())
    r, B, C = (x @ W_x).split([8, 8, 8], -1)
    args = (x, r @ W_dt, layer.A_log.detach(), B.unsqueeze(1), C.unsqueeze(1), cu, layer.D.detach(), z, layer.dt_bias.detach())
    o = ref.scan(*args)["y"][0]
    stream64 = d(stream) + o @ W_out
    # and back
    n = ref.norm_bwd(stream64, norm, dy, dh=dh)
    dout = n["dresidual"][0]
    g = ref.scan(*args, dy=dout @ W_out.t())
    dr = g["ddt"][0] @ W_dt.t()
    dxp = torch.cat([dr, g["dB"][0].flatten(1), g["dC"][0].flatten(1)], 1)
    dx = g["dx"][0] + dxp @ W_x.t()
    _, _, c, _ = ref.conv(x0, layer.conv.detach(), cu, layer.bias.detach(), dy=dx)
    want = {"w_out": o.t() @ dout, "w_x": x.t() @ dxp, "w_dt": r.t() @ g["ddt"][0], "conv": c["dw"], "bias": c["db"],
            "w_in": d(u).t() @ torch.cat([c["dx"], g["dz"][0]], 1), "A_log": g["dA_log"][0], "dt_bias": g["ddt_bias"][0],
            "D": g["dD"][0]}
    # each operator is off by at most 2^-12 of its terms, three of them and four products of fp32 by 2^-10; their
    # terms are at most four times their sums in norm here
    for name, value in want.items():
        got = getattr(layer, name).grad.double()
        assert float((got - value).norm() / value.norm()) < 2.0 ** -8, name
    for got, value in ((w.grad, n["dweight"][0]), (s.grad, n["dresidual"][0])):
        assert float((got.double() - value).norm() / value.norm()) < 2.0 ** -8

