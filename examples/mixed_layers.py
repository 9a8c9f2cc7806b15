"""Two layers of a mixed model trained and served with the library: a gated delta rule layer (short
convolution of q, k and v, the rule, the gated norm) and a selective layer (short convolution, selective
scan), with a residual norm ahead of each.

    PYTHONPATH=. python examples/mixed_layers.py
"""
import numpy as np
import torch

import chunked_gated_delta_06_gb300 as gdn

D, W = 128, 4


def _weights(seed, device, dtype):
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def weight(*shape, scale=None, kind=dtype):
        w = torch.randn(*shape, generator=g, device=device) * (shape[0] ** -0.5 if scale is None else scale)
        return w.to(kind).requires_grad_()
    return weight


class DeltaLayer:
    """x [T, hidden] -> [T, hidden]: q and k of H heads, v and the gate z of HV heads."""

    def __init__(self, hidden, H, HV, seed=0, device="cuda"):
        self.H, self.HV = H, HV
        weight, f32 = _weights(seed, device, torch.bfloat16), torch.float32
        self.qkv = (2 * H + HV) * D
        self.w_in, self.w_out = weight(hidden, self.qkv + HV * D), weight(HV * D, hidden)
        self.w_ab = weight(hidden, 2 * HV)
        self.conv = weight(self.qkv, W, scale=W ** -0.5, kind=f32)
        self.norm = weight(D, scale=0.1, kind=f32)
        self.log_rate = weight(HV, scale=0.1, kind=f32)

    def parameters(self):
        return [self.w_in, self.w_out, self.w_ab, self.conv, self.norm, self.log_rate]

    def split(self, u, ab):
        """q, k, v of the convolution's output; the log decay and beta."""
        q, k, v = (t.unflatten(-1, (-1, D)).contiguous() for t in u.split([self.H * D, self.H * D, self.HV * D], -1))
        a, b = ab.float().chunk(2, -1)
        return q, k, v, (-self.log_rate.exp() * torch.nn.functional.softplus(a)).contiguous(), b.sigmoid().contiguous()

    def finish(self, o, z):
        y = gdn.rms_norm(o, self.norm, z=z.unflatten(-1, (-1, D)), offset=1.0)
        return y.flatten(-2) @ self.w_out

    def train(self, x, cu, cu_host):
        u, ab = x @ self.w_in, x @ self.w_ab
        mixed, z = u.split([self.qkv, self.HV * D], -1)
        mixed, _ = gdn.short_conv(mixed, self.conv, cu_seqlens=cu, cu_seqlens_cpu=cu_host)
        q, k, v, g, beta = self.split(mixed, ab)
        o, _ = gdn.chunk_gated_delta_rule(q, k, v, g, beta, cu_seqlens=cu, cu_seqlens_cpu=cu_host)
        return self.finish(o, z)

    def pools(self, slots, device="cuda"):
        return (torch.zeros(slots, self.qkv, W - 1, device=device, dtype=torch.bfloat16),
                torch.zeros(slots, self.HV, D, D, device=device))

    @torch.no_grad()
    def prefill(self, x, cu, cu_host, pools, slots, resume):
        u, ab = x @ self.w_in, x @ self.w_ab
        mixed, z = u.split([self.qkv, self.HV * D], -1)
        mixed = gdn.short_conv_prefill_paged(mixed, self.conv, cu_host, cu, pools[0], slots, resume)
        q, k, v, g, beta = self.split(mixed, ab)
        return self.finish(gdn.chunk_prefill_paged(q, k, v, g, beta, cu_host, cu, pools[1], slots, resume), z)

    @torch.no_grad()
    def step(self, x, pools, slots):
        u, ab = x @ self.w_in, x @ self.w_ab
        mixed, z = u.split([self.qkv, self.HV * D], -1)
        mixed = gdn.short_conv_step(mixed, self.conv, pools[0], slots)
        q, k, v, g, beta = self.split(mixed, ab)
        return self.finish(gdn.decode_step(q, k, v, g, beta, pools[1], slots), z)


class SelectiveLayer:
    """x [T, hidden] -> [T, hidden]: `channels` channels of Ns states each, steps from `rank` features."""

    def __init__(self, hidden, channels, Ns=16, rank=32, seed=1, device="cuda", dtype=torch.bfloat16):
        weight, f32 = _weights(seed, device, dtype), torch.float32
        self.channels, self.Ns, self.rank = channels, Ns, rank
        self.w_in, self.w_out = weight(hidden, 2 * channels), weight(channels, hidden)
        self.w_x, self.w_dt = weight(channels, rank + 2 * Ns), weight(rank, channels)
        self.conv, self.bias = weight(channels, W, scale=W ** -0.5, kind=f32), weight(channels, scale=0.1, kind=f32)
        rates = torch.log(torch.arange(1, Ns + 1, device=device, dtype=f32)).repeat(channels, 1)
        steps = torch.exp(torch.linspace(-6.9, -2.3, channels, device=device))
        self.A_log, self.dt_bias = rates.requires_grad_(), torch.log(torch.expm1(steps)).requires_grad_()
        self.D = torch.ones(channels, device=device).requires_grad_()

    def parameters(self):
        return [self.w_in, self.w_out, self.w_x, self.w_dt, self.conv, self.bias, self.A_log, self.dt_bias, self.D]

    def terms(self, x):
        """dt, B and C of the convolution's output."""
        r, B, C = (x @ self.w_x).split([self.rank, self.Ns, self.Ns], -1)
        return r @ self.w_dt, B.unsqueeze(1), C.unsqueeze(1)

    def train(self, u, cu, cu_host):
        x, z = (u @ self.w_in).split([self.channels, self.channels], -1)
        x, _ = gdn.short_conv(x, self.conv, self.bias, cu_seqlens=cu, cu_seqlens_cpu=cu_host)
        dt, B, C = self.terms(x)
        y, _ = gdn.selective_scan(x, dt, self.A_log, B, C, D=self.D, z=z, dt_bias=self.dt_bias, cu_seqlens=cu,
                                  cu_seqlens_cpu=cu_host)
        return y @ self.w_out

    def pools(self, slots, device="cuda"):
        return (torch.zeros(slots, self.channels, W - 1, device=device, dtype=self.w_in.dtype),
                torch.zeros(slots, self.channels, self.Ns, device=device))

    @torch.no_grad()
    def prefill(self, u, cu, cu_host, pools, slots, resume):
        x, z = (u @ self.w_in).split([self.channels, self.channels], -1)
        x = gdn.short_conv_prefill_paged(x, self.conv, cu_host, cu, pools[0], slots, resume, bias=self.bias)
        dt, B, C = self.terms(x)
        y = gdn.selective_scan_prefill_paged(x, dt, self.A_log, B, C, cu_host, cu, pools[1], slots, resume, D=self.D, z=z,
                                             dt_bias=self.dt_bias)
        return y @ self.w_out

    @torch.no_grad()
    def step(self, u, pools, slots):
        x, z = (u @ self.w_in).split([self.channels, self.channels], -1)
        x = gdn.short_conv_step(x, self.conv, pools[0], slots, bias=self.bias)
        dt, B, C = self.terms(x)
        y = gdn.selective_scan_step(x, dt, self.A_log, B, C, pools[1], slots, D=self.D, z=z, dt_bias=self.dt_bias)
        return y @ self.w_out


class Model:
    """The layers with a residual norm ahead of each and one behind the last."""

    def __init__(self, hidden, layers, device="cuda"):
        self.layers = layers
        self.norms = [torch.zeros(hidden, device=device, requires_grad=True) for _ in range(len(layers) + 1)]

    def parameters(self):
        return self.norms + [p for layer in self.layers for p in layer.parameters()]

    def run(self, x, call):
        h = x.float()
        y = gdn.rms_norm(h, self.norms[0], offset=1.0).to(x.dtype)
        for layer, norm in zip(self.layers, self.norms[1:]):
            y, h = gdn.rms_norm(call(layer, y), norm, residual=h, offset=1.0)
        return y


def packed(lens, device="cuda"):
    cu_host = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu_host, torch.from_numpy(cu_host).to(device)


def main(hidden=256, prompts=(150, 37), answer=5):
    model = Model(hidden, [DeltaLayer(hidden, 2, 4), SelectiveLayer(hidden, 512)])
    lens = [n + answer for n in prompts]
    cu_host, cu = packed(lens)
    x = torch.randn(int(cu_host[-1]), hidden, device="cuda").to(torch.bfloat16)

    # a training step
    y = model.run(x, lambda layer, u: layer.train(u, cu, cu_host))
    loss = y.float().square().mean()
    loss.backward()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in model.parameters())

    # the same sequences served: a prefill of the prompts, then a step for each further token
    pools = {layer: layer.pools(len(lens) + 1) for layer in model.layers}
    slots = torch.arange(1, len(lens) + 1, dtype=torch.int32, device="cuda")
    fresh = torch.zeros_like(slots)
    pc_host, pc = packed(prompts)
    out = torch.empty_like(y)
    with torch.no_grad():
        at = torch.cat([torch.arange(a, a + n) for a, n in zip(cu_host, prompts)]).cuda()
        out[at] = model.run(x[at], lambda layer, u: layer.prefill(u, pc, pc_host, pools[layer], slots, fresh))
        for j in range(answer):
            at = torch.tensor([a + n + j for a, n in zip(cu_host, prompts)], device="cuda")
            out[at] = model.run(x[at], lambda layer, u: layer.step(u, pools[layer], slots))
    off = float((out.float() - y.detach().float()).norm() / y.detach().float().norm())
    print("loss %.4f, served and trained outputs differ by %.2e" % (float(loss.detach()), off))
    return off


if __name__ == "__main__":
    main()
