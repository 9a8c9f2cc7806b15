"""A decay-only linear-attention layer trained and served with the library: rotary positions,
the packed forward and its gradient, a paged prefill and single-token steps over its slots.

    PYTHONPATH=. python examples/linear_layer.py
"""
import numpy as np
import torch

import chunked_gated_delta_06_gb300 as gdn

D = 128


class LinearLayer:
    """x [T, hidden] -> [T, hidden]: q and k of H heads (half of each rotated), v of HV heads,
    one decay for each value head."""

    def __init__(self, hidden, H, HV, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.H, self.HV = H, HV

        def weight(a, b):
            w = torch.randn(a, b, generator=g, device=device) * a ** -0.5
            return w.to(torch.bfloat16).requires_grad_()
        self.wq, self.wk, self.wv = weight(hidden, H * D), weight(hidden, H * D), weight(hidden, HV * D)
        self.wo = weight(HV * D, hidden)
        # geometric slopes; the decay is a constant of the layer
        self.log_decay = -torch.exp2(-8.0 * torch.arange(1, HV + 1, device=device) / HV).float()
        self.freq = gdn.rope_frequencies(D // 2, device=device)   # 64 of a head's 128 elements turn

    def parameters(self):
        return [self.wq, self.wk, self.wv, self.wo]

    def project(self, x):
        q, k, v = (x @ w for w in (self.wq, self.wk, self.wv))
        return (torch.nn.functional.silu(q).view(-1, self.H, D), torch.nn.functional.silu(k).view(-1, self.H, D),
                v.view(-1, self.HV, D))

    def train(self, x, positions, cu, cu_host):
        """Packed sequences, differentiable."""
        q, k, v = self.project(x)
        q, k = gdn.rotary(q, k, positions, self.freq)
        o, _ = gdn.linear_attention(q, k, v, self.log_decay, cu_seqlens=cu, cu_seqlens_cpu=cu_host)
        return o.reshape(len(x), -1) @ self.wo

    @torch.no_grad()
    def prefill(self, x, positions, cu, cu_host, pool, slots, resume=None):
        """Prompts (or further parts of them), their states left in the pool's slots."""
        q, k, v = self.project(x)
        gdn.rope(q, k, positions, self.freq, inplace=True)
        o = gdn.linear_attn_prefill_paged(q, k, v.contiguous(), self.log_decay, cu_host, cu, pool, slots, resume)
        return o.reshape(len(x), -1) @ self.wo

    @torch.no_grad()
    def step(self, x, positions, pool, slots):
        """One token for each row."""
        q, k, v = self.project(x)
        gdn.rope(q, k, positions, self.freq, inplace=True)
        o = gdn.linear_attn_step(q, k, v.contiguous(), self.log_decay, pool, slots)
        return o.reshape(len(x), -1) @ self.wo


def packed(lens, device="cuda"):
    """Sequence boundaries (host and device) and each token's position."""
    cu_host = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(device)
    return cu_host, torch.from_numpy(cu_host).to(device), positions


def main(hidden=512, H=4, HV=8, prompts=(300, 37), answer=5):
    layer = LinearLayer(hidden, H, HV)
    lens = [n + answer for n in prompts]
    cu_host, cu, positions = packed(lens)
    x = torch.randn(int(cu_host[-1]), hidden, device="cuda").to(torch.bfloat16)

    # a training step
    y = layer.train(x, positions, cu, cu_host)
    loss = y.float().square().mean()
    loss.backward()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in layer.parameters())

    # the same sequences served: a prefill of the prompts, then a step for each further token
    pool = torch.zeros(len(lens) + 1, HV, D, D, device="cuda")
    slots = torch.arange(1, len(lens) + 1, dtype=torch.int32, device="cuda")
    rows = [torch.arange(a, a + n) for a, n in zip(cu_host, prompts)]
    pc_host, pc, ppos = packed(prompts)
    out = torch.empty_like(y)
    at = torch.cat(rows).cuda()
    out[at] = layer.prefill(x[at], ppos, pc, pc_host, pool, slots,
                            resume=torch.zeros(len(lens), dtype=torch.int32, device="cuda"))
    for j in range(answer):
        at = torch.tensor([a + n + j for a, n in zip(cu_host, prompts)], device="cuda")
        out[at] = layer.step(x[at], positions[at].contiguous(), pool, slots)
    off = float((out.float() - y.detach().float()).norm() / y.detach().float().norm())
    print("loss %.4f, served and trained outputs differ by %.2e" % (float(loss.detach()), off))
    return off


if __name__ == "__main__":
    main()
