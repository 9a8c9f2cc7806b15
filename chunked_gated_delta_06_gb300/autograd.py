"""The chunk path as a differentiable PyTorch function, with the call shape of the
pages' op ("[Cake 1/13] gdn: chunked gated delta rule, det and fast, with KCP and
FLA-CP", API and flags: chunk_gated_delta_rule(q, k, v, g, beta, scale,
initial_state, output_final_state, cu_seqlens, cu_seqlens_cpu, ...), packed B = 1,
in-kernel q/k L2 norm, the recompute-state option).

Argument marshalling only: the forward calls gdn_chunk_fwd and the backward
gdn_chunk_bwd through the C ABI (binding.chunk_fwd / chunk_bwd).
"""
from __future__ import annotations

import numpy as np

from . import binding, linear


def _final(name, grads, inputs):
    """The gradients of a fused backward, which are not differentiable themselves: where the caller
    records a graph of them (create_graph), differentiating it raises instead of taking them for
    constants.  inputs: what they depend on."""
    import torch
    inputs = [x for x in inputs if x is not None and x.requires_grad]
    if not torch.is_grad_enabled() or not inputs:
        return grads

    class Final(torch.autograd.Function):
        @staticmethod
        def forward(ctx, count, *tensors):
            return tensors[:count]

        @staticmethod
        def backward(ctx, *unused):
            raise RuntimeError("the gradients of %s cannot be differentiated once more" % name)

    there = [x for x in grads if x is not None]
    marked = iter(Final.apply(len(there), *there, *inputs))
    return tuple(None if x is None else next(marked) for x in grads)


def _function():
    import torch

    class ChunkGatedDeltaRule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, g, beta, initial_state, cu_host, cu_dev, scale, output_final_state,
                    recompute_state):
            ctx.set_materialize_grads(False)
            o, ht, c = binding.chunk_fwd(q, k, v, g, beta, cu_host, cu_dev, scale=scale,
                                         initial_state=initial_state,
                                         output_final_state=output_final_state,
                                         for_backward=not recompute_state)
            ctx.gdn = c
            ctx.has_h0 = initial_state is not None
            ctx.save_for_backward(q, k, v, g, beta, initial_state)
            return o, ht

        @staticmethod
        def backward(ctx, d_o, d_ht):
            q, k, v, g, beta, h0 = ctx.saved_tensors
            if d_o is None:
                d_o = torch.zeros((q.shape[0], v.shape[1], v.shape[2]), dtype=torch.bfloat16,
                                  device=q.device)
            gr = binding.chunk_bwd(ctx.gdn, q, k, v, g, beta, d_o.to(torch.bfloat16).contiguous(),
                                   d_final_state=None if d_ht is None else d_ht.float().contiguous(),
                                   initial_state=h0, want_dh0=ctx.has_h0)
            grads = _final("chunk_gated_delta_rule", [gr[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0")],
                           (q, k, v, g, beta, h0, d_o, d_ht))
            return (*grads, None, None, None, None, None)

    return ChunkGatedDeltaRule


_FN = None


def chunk_gated_delta_rule(q, k, v, g, beta, scale=None, initial_state=None, output_final_state=False,
                           cu_seqlens=None, cu_seqlens_cpu=None, recompute_state=False):
    """o [B=1, T, HV, V] (and the final state [N, HV, K, V] when output_final_state).

    q, k: bf16 [1, T, H, 128] or [T, H, 128]; v: bf16 [.., T, HV, 128]; g: fp32 [.., T, HV];
    beta: bf16 or fp32 [.., T, HV]; initial_state: fp32 [N, HV, 128, 128] or None;
    cu_seqlens: int32 device [N + 1] (default: one sequence), cu_seqlens_cpu: the same
    boundaries on the host (read from cu_seqlens when not given: one device-to-host copy).
    recompute_state: the backward rebuilds w, u, h and v_new instead of keeping them."""
    import torch
    global _FN
    if _FN is None:
        _FN = _function()
    batched = q.dim() == 4
    if batched:
        if q.shape[0] != 1:
            raise ValueError("packed sequences only: B must be 1 (use cu_seqlens)")
        q, k, v, g, beta = q[0], k[0], v[0], g[0], beta[0]
    T = q.shape[0]
    if cu_seqlens is None:
        cu_seqlens = torch.tensor([0, T], dtype=torch.int32, device=q.device)
    if cu_seqlens_cpu is None:
        cu_seqlens_cpu = cu_seqlens.cpu()
    cu_host = np.asarray(cu_seqlens_cpu.cpu() if hasattr(cu_seqlens_cpu, "cpu") else cu_seqlens_cpu,
                         dtype=np.int32)
    o, ht = _FN.apply(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), beta.contiguous(),
                      initial_state, cu_host, cu_seqlens.to(torch.int32).contiguous(), scale,
                      output_final_state, recompute_state)
    if batched:
        o = o.unsqueeze(0)
    return o, ht


def _linear_function():
    import torch

    class LinearAttention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, log_decay, initial_state, cu_host, cu_dev, scale, output_final_state):
            ctx.set_materialize_grads(False)
            ctx.cu_host, ctx.scale = cu_host.copy(), scale   # (the caller may reuse its buffer)
            ctx.save_for_backward(q, k, v, log_decay, initial_state, cu_dev)
            return linear.linear_attn_fwd(q, k, v, log_decay, cu_host, cu_dev, scale=scale,
                                           initial_state=initial_state,
                                           output_final_state=output_final_state)

        @staticmethod
        def backward(ctx, d_o, d_ht):
            q, k, v, log_decay, h0, cu_dev = ctx.saved_tensors
            if d_o is None:
                d_o = torch.zeros_like(v)
            gr = linear.linear_attn_bwd(q, k, v, log_decay, d_o.to(torch.bfloat16).contiguous(), ctx.cu_host,
                                         cu_dev, scale=ctx.scale, initial_state=h0,
                                         d_final_state=None if d_ht is None else d_ht.float().contiguous(),
                                         want_dh0=h0 is not None)
            dq, dk, dv, dh0 = _final("linear_attention", [gr[n] for n in ("dq", "dk", "dv", "dh0")],
                                     (q, k, v, h0, d_o, d_ht))
            return dq, dk, dv, None, dh0, None, None, None, None

    return LinearAttention


def _rotary_function():
    import torch

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, positions, freq, layout, mscale, transposed):
            ctx.args = (layout, mscale, transposed)
            ctx.save_for_backward(positions, freq)
            return linear.rope(q, k, positions, freq, layout=layout, mscale=mscale, backward=transposed)

        @staticmethod
        def backward(ctx, dq, dk):
            # the other direction of the same operator, so that it has a gradient of its own
            layout, mscale, transposed = ctx.args
            dq, dk = Rotary.apply(dq.contiguous(), None if dk is None else dk.contiguous(), *ctx.saved_tensors,
                                  layout, mscale, not transposed)
            return dq, dk, None, None, None, None, None

    return Rotary


_LINEAR = _ROTARY = None


def linear_attention(q, k, v, log_decay, scale=None, initial_state=None, output_final_state=False,
                     cu_seqlens=None, cu_seqlens_cpu=None):
    """Differentiable linear attention with a decay for each head, in the call shape of
    chunk_gated_delta_rule: o (and the final state [N, HV, K, V] when output_final_state).

    log_decay: fp32 [HV], <= 0, a constant of the layer: asking for its gradient is refused, as is
    differentiating the gradients once more."""
    global _LINEAR
    if log_decay.requires_grad:
        raise ValueError("log_decay has no gradient: pass it detached")
    if _LINEAR is None:
        _LINEAR = _linear_function()
    import torch
    batched = q.dim() == 4
    if batched:
        if q.shape[0] != 1:
            raise ValueError("packed sequences only: B must be 1 (use cu_seqlens)")
        q, k, v = q[0], k[0], v[0]
    if cu_seqlens is None:
        cu_seqlens = torch.tensor([0, q.shape[0]], dtype=torch.int32, device=q.device)
    if cu_seqlens_cpu is None:
        cu_seqlens_cpu = cu_seqlens.cpu()
    cu_host = np.asarray(cu_seqlens_cpu.cpu() if hasattr(cu_seqlens_cpu, "cpu") else cu_seqlens_cpu,
                         dtype=np.int32)
    o, ht = _LINEAR.apply(q.contiguous(), k.contiguous(), v.contiguous(), log_decay.contiguous(),
                          initial_state, cu_host, cu_seqlens.to(torch.int32).contiguous(), scale,
                          output_final_state)
    return (o.unsqueeze(0) if batched else o), ht


def rotary(q, k, positions, freq, layout="half", mscale=1.0):
    """Differentiable rotary positions of q [T, Hq, D] and k [T, Hk, D] or None (linear.rope), to
    any order.  freq is a constant of the model: asking for its gradient is refused."""
    global _ROTARY
    import torch
    if freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("freq has no gradient: pass it detached")
    if _ROTARY is None:
        _ROTARY = _rotary_function()
    return _ROTARY.apply(q.contiguous(), None if k is None else k.contiguous(), positions, freq, layout, mscale,
                         False)
