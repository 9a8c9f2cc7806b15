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

from . import binding, linear, mixer


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
            cu_host = cu_host.copy()   # (the backward reads it again, and the caller may reuse its buffer)
            o, ht, c = binding.chunk_fwd(q, k, v, g, beta, cu_host, cu_dev, scale=scale,
                                         initial_state=initial_state,
                                         output_final_state=output_final_state,
                                         for_backward=not recompute_state)
            ctx.gdn = c
            ctx.has_h0 = initial_state is not None
            ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_dev)
            return o, ht

        @staticmethod
        def backward(ctx, d_o, d_ht):
            q, k, v, g, beta, h0, _ = ctx.saved_tensors   # (the offsets too: they must not have changed)
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
    boundaries on the host (either is copied from the other when not given).
    recompute_state: the backward rebuilds w, u, h and v_new instead of keeping them."""
    global _FN
    if _FN is None:
        _FN = _function()
    batched = q.dim() == 4
    if batched:
        q, k, v, g, beta = _one_batch(q, k, v, g, beta)
    cu_host, cu_dev = _offsets(q.shape[0], q.device, cu_seqlens, cu_seqlens_cpu)
    o, ht = _FN.apply(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), beta.contiguous(),
                      initial_state, cu_host, cu_dev, scale, output_final_state, recompute_state)
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
    batched = q.dim() == 4
    if batched:
        q, k, v = _one_batch(q, k, v)
    cu_host, cu_dev = _offsets(q.shape[0], q.device, cu_seqlens, cu_seqlens_cpu)
    o, ht = _LINEAR.apply(q.contiguous(), k.contiguous(), v.contiguous(), log_decay.contiguous(),
                          initial_state, cu_host, cu_dev, scale, output_final_state)
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


def _aligned(t):
    """t, or a copy of it, dense and from 16 bytes on (the gradients that reach a function may be parts of
    a wider tensor)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _mixer_functions():
    import torch

    class ShortConv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, initial_state, cu_host, cu_dev, activation, output_final_state):
            ctx.set_materialize_grads(False)
            ctx.cu_host, ctx.activation = cu_host.copy(), activation
            ctx.save_for_backward(x, weight, bias, initial_state, cu_dev)
            return mixer.short_conv_fwd(x, weight, cu_host, cu_dev, bias=bias, activation=activation,
                                        initial_state=initial_state, output_final_state=output_final_state)

        @staticmethod
        def backward(ctx, dy, dht):
            x, weight, bias, h0, cu_dev = ctx.saved_tensors
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy
            gr = mixer.short_conv_bwd(x, weight, _aligned(dy), ctx.cu_host, cu_dev, bias=bias,
                                      activation=ctx.activation, initial_state=h0, d_final_state=_aligned(dht),
                                      want_dh0=h0 is not None)
            grads = _final("short_conv", [gr[n] for n in ("dx", "dw", "dbias", "dh0")],
                           (x, weight, bias, h0, dy, dht))
            return (*grads, None, None, None, None)

    class SelectiveScan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, dt, A_log, B, C, D, z, dt_bias, initial_state, cu_host, cu_dev, output_final_state):
            ctx.set_materialize_grads(False)
            ctx.cu_host = cu_host.copy()
            ctx.save_for_backward(x, dt, A_log, B, C, D, z, dt_bias, initial_state, cu_dev)
            return mixer.selective_scan_fwd(x, dt, A_log, B, C, cu_host, cu_dev, D=D, z=z, dt_bias=dt_bias,
                                            initial_state=initial_state, output_final_state=output_final_state)

        @staticmethod
        def backward(ctx, dy, dht):
            *inputs, cu_dev = ctx.saved_tensors
            x, dt, A_log, B, C, D, z, dt_bias, h0 = inputs
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy
            gr = mixer.selective_scan_bwd(x, dt, A_log, B, C, _aligned(dy), ctx.cu_host, cu_dev, D=D, z=z,
                                          dt_bias=dt_bias, initial_state=h0, d_final_state=_aligned(dht),
                                          want_dh0=h0 is not None)
            names = ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
            grads = _final("selective_scan", [gr[n] for n in names], (*inputs, dy, dht))
            return (*grads, None, None, None)

    class RmsNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, z, residual, scale, gate, eps, offset):
            ctx.set_materialize_grads(False)
            y, h = mixer.rms_norm_fwd(x, weight, z=z, residual=residual, scale=scale, gate=gate, eps=eps, offset=offset)
            ctx.args, ctx.kind = dict(gate=gate, eps=eps, offset=offset, residual=residual is not None), x.dtype
            ctx.save_for_backward(x if h is None else h, weight, z, scale, x if scale is not None else None)
            return y, h

        @staticmethod
        def backward(ctx, dy, dh):
            h, weight, z, scale, x = ctx.saved_tensors
            dy = torch.zeros(h.shape, dtype=ctx.kind, device=h.device) if dy is None else dy
            gr = mixer.rms_norm_bwd(h, weight, _aligned(dy), z=z, dh=_aligned(dh), scale=scale, x=x, **ctx.args)
            grads = _final("rms_norm", [gr[n] for n in ("dx", "dweight", "dz", "dresidual", "dscale")],
                           (h, weight, z, scale, x, dy, dh))
            return (*grads, None, None, None)

    return ShortConv, SelectiveScan, RmsNorm


_MIXER = None


def _mixer(which):
    global _MIXER
    if _MIXER is None:
        _MIXER = _mixer_functions()
    return _MIXER[which]


def _dense_rows(t):
    """t, or a copy of it whose rows are dense."""
    if t is None or t.is_contiguous():
        return t
    width = 1
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and s != width:
            return t.contiguous()
        width *= n
    return t if t.stride(0) >= width else t.contiguous()


def _offsets(T, device, cu_seqlens, cu_seqlens_cpu):
    """The sequences' offsets on the host and on the device, either from the other where one is not given; one
    sequence of T tokens without both."""
    import torch
    if cu_seqlens_cpu is None:
        cu_seqlens_cpu = np.array([0, T], dtype=np.int32) if cu_seqlens is None else cu_seqlens.cpu()
    cu_host = np.asarray(cu_seqlens_cpu.cpu() if hasattr(cu_seqlens_cpu, "cpu") else cu_seqlens_cpu, dtype=np.int32)
    if cu_seqlens is None:
        cu_seqlens = torch.tensor(cu_host, dtype=torch.int32, device=device)
    return cu_host, cu_seqlens.to(torch.int32).contiguous()


def _one_batch(*tensors):
    if any(t is not None and t.shape[0] != 1 for t in tensors):
        raise ValueError("packed sequences only: B must be 1 (use cu_seqlens)")
    return [None if t is None else t[0] for t in tensors]


def _float(t):
    return None if t is None else t.float().contiguous()


def short_conv(x, weight, bias=None, activation="silu", initial_state=None, output_final_state=False,
               cu_seqlens=None, cu_seqlens_cpu=None):
    """Differentiable short causal convolution of packed sequences: y like x (and the final state [N, C,
    W - 1] when output_final_state).  x: [T, C] or [1, T, C], bf16 or fp32, rows may lie apart; weight [C, W]
    and bias [C] of any floating type (computed with in fp32); activation: "silu" or None."""
    batched = x.dim() == 3
    if batched:
        (x,) = _one_batch(x)
    cu_host, cu_dev = _offsets(x.shape[0], x.device, cu_seqlens, cu_seqlens_cpu)
    y, ht = _mixer(0).apply(_dense_rows(x), _float(weight), _float(bias), _aligned(initial_state), cu_host, cu_dev,
                            activation, output_final_state)
    return (y.unsqueeze(0) if batched else y), ht


def selective_scan(x, dt, A_log, B, C, D=None, z=None, dt_bias=None, initial_state=None, output_final_state=False,
                   cu_seqlens=None, cu_seqlens_cpu=None):
    """Differentiable selective state space scan of packed sequences: y like x (and the final state fp32
    [N, channels, state_dim] when output_final_state).  x, dt, z: [T, channels] or [1, T, channels]; B, C:
    [.., T, groups, state_dim]; rows may lie apart; A_log [channels, state_dim], D and dt_bias [channels] of
    any floating type (computed with in fp32)."""
    batched = x.dim() == 3
    if batched:
        x, dt, B, C, z = _one_batch(x, dt, B, C, z)
    cu_host, cu_dev = _offsets(x.shape[0], x.device, cu_seqlens, cu_seqlens_cpu)
    y, ht = _mixer(1).apply(_dense_rows(x), _dense_rows(dt), _float(A_log), _dense_rows(B), _dense_rows(C), _float(D),
                            _dense_rows(z), _float(dt_bias), _aligned(initial_state), cu_host, cu_dev,
                            output_final_state)
    return (y.unsqueeze(0) if batched else y), ht


def rms_norm(x, weight, z=None, residual=None, scale=None, gate="silu", eps=1e-6, offset=0.0):
    """Differentiable norm of rows with its gate and residual: y = h / rms(h) (offset + weight) act(z), with
    h = residual + scale x returned as well, (y, h), where there is a residual.  x, z, residual: [..., dim];
    weight and scale [dim] of any floating type (computed with in fp32)."""
    y, h = _mixer(2).apply(_aligned(x), _aligned(_float(weight)), _aligned(z), _aligned(residual),
                           _aligned(_float(scale)), gate, eps, offset)
    return y if residual is None else (y, h)
