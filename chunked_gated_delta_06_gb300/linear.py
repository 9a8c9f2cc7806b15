"""The decay-only linear attention and the rotary positions on torch tensors: argument checks and
marshalling only, every step of the computation runs in libgdn's CUDA kernels.

These calls are also made for a few tokens at a time, where the time is the host's: the checks
compare whole shapes, gdn_problem is packed in one go, and the workspace is asked for only when
the library says that the call needs one.
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np

from . import binding
from .binding import GDN_ERR_WORKSPACE_TOO_SMALL, GDN_OK, GdnError



def _struct_of(layout):
    """A ctypes structure's fields, in their order, to be packed in one go."""
    codes = "".join(t._type_ if isinstance(t._type_, str) else "P" for _, t in layout._fields_)
    return struct.Struct("@%s%dx" % (codes, ctypes.sizeof(layout) - struct.calcsize("@" + codes)))


_PROBLEM = _struct_of(binding.GdnProblem)
_ROPE_SCALING = {"none": binding.GDN_ROPE_SCALE_NONE, "linear": binding.GDN_ROPE_SCALE_LINEAR,
                 "parts": binding.GDN_ROPE_SCALE_PARTS}
_ROPE_LAYOUT = {"half": binding.GDN_ROPE_HALF, "interleaved": binding.GDN_ROPE_INTERLEAVED}

torch = None
_raw_stream = _current_device = None


def _ready():
    """The library; torch is imported by the first call, not with the package."""
    global torch, _raw_stream, _current_device
    if torch is None:
        import torch as module
        torch = module
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _current_device = torch._C._cuda_getDevice
    return binding._lib or binding.lib()


def _device(q):
    """The device of a call: q's, which must be the current one (the library launches there)."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a contiguous CUDA tensor")
    if dev != _current_device():
        raise ValueError("q is on cuda:%d, which is not the current device" % dev)
    return dev


def _need(t, name, dtype, shape, dev):
    """Refuse a tensor the kernels would misread: they take dense tensors of one dtype on the
    call's device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, shape, tuple(t.shape)))
    if t.is_cuda and t.get_device() != dev:
        raise ValueError("%s is on cuda:%d, not on q's device" % (name, t.get_device()))
    raise ValueError("%s must be a contiguous CUDA tensor" % name)


def _maybe(t, name, dtype, shape, dev):
    return None if t is None else _need(t, name, dtype, shape, dev)


def _status(t, dev):
    if t is None:
        return None
    if t.dtype is not torch.int32 or not t.is_cuda or t.numel() < 1:
        raise TypeError("a device status is an int32 CUDA tensor")
    if t.get_device() != dev:
        raise ValueError("a device status must be on q's device")
    return t.data_ptr()


def _inputs(q, k, v, log_decay):
    """(T, H, K, HV, V), the four addresses and the device."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, 128]")
    bf = torch.bfloat16
    T, H, K = shape = q.shape
    _, HV, V = v.shape
    dev = _device(q)
    return (T, H, K, HV, V), (_need(q, "q", bf, shape, dev), _need(k, "k", bf, shape, dev),
                              _need(v, "v", bf, (T, HV, V), dev),
                              _need(log_decay, "log_decay", torch.float32, (HV,), dev)), dev


def _problem(dims, cu_host, cu_dev, scale, status, segments, dev):
    """gdn_problem as bytes, the array it points at (to be kept alive), and N."""
    T, H, K, HV, V = dims
    cu = cu_host
    if type(cu) is not np.ndarray or cu.dtype != np.int32 or not cu.flags.c_contiguous:
        cu = np.ascontiguousarray(np.asarray(cu_host, dtype=np.int32))
    N = len(cu) - 1
    if N < 1 or cu[N] != T:
        raise ValueError("cu_host must end with the number of tokens, %d" % T)
    # (in the order of GdnProblem)
    return _PROBLEM.pack(N, T, H, HV, K, V, scale or 0.0, 0, cu.__array_interface__["data"][0],
                         _need(cu_dev, "cu_dev", torch.int32, (N + 1,), dev), _status(status, dev) or 0, segments), cu, N


def _call(fn, name, problem, mode, args, workspace, dev):
    """fn(problem, *args, workspace, bytes, stream): without a workspace first, which most short
    calls do not need."""
    stream = _raw_stream(dev)
    if workspace is None:
        st = fn(problem, *args, None, 0, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on q's device")
    else:
        st = fn(problem, *args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), stream)
    if st == GDN_ERR_WORKSPACE_TOO_SMALL:
        n = binding._lib.gdn_linear_attn_workspace_bytes(problem, mode)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        st = fn(problem, *args, workspace.data_ptr(), n, stream)
    if st != GDN_OK:
        raise GdnError(st, name)


def linear_attn_fwd(q, k, v, log_decay, cu_host, cu_dev, scale=None, initial_state=None,
                    output_final_state=True, workspace=None, device_status=None, scan_segment_chunks=0):
    """gdn_linear_attn_fwd on torch tensors.  Returns (o, final_state or None).

    q, k: bf16 [T, H, 128]; v: bf16 [T, HV, 128]; log_decay: fp32 [HV]; cu_host / cu_dev: the
    int32 sequence boundaries on the host and on the device; states fp32 [N, HV, K, V].
    scan_segment_chunks: the problem field of that name, in chunks of 128 tokens."""
    L = _ready()
    dims, inputs, dev = _inputs(q, k, v, log_decay)
    p, keep, N = _problem(dims, cu_host, cu_dev, scale, device_status, scan_segment_chunks, dev)
    shape = (N, dims[3], 128, 128)
    h0 = _maybe(initial_state, "initial_state", torch.float32, shape, dev)
    o = torch.empty_like(v)
    ht = torch.empty(shape, dtype=torch.float32, device=q.device) if output_final_state else None
    _call(L.gdn_linear_attn_fwd, "gdn_linear_attn_fwd", p, 0,
          (*inputs, h0, o.data_ptr(), None if ht is None else ht.data_ptr()), workspace, dev)
    return o, ht


def linear_attn_prefill_paged(q, k, v, log_decay, cu_host, cu_dev, state_pool, state_indices,
                              has_initial_state=None, scale=None, device_status=None, workspace=None,
                              problem_status=None, scan_segment_chunks=0):
    """gdn_linear_attn_prefill_paged on torch tensors (state_pool updated in place; slots and
    status words as in chunk_prefill_paged).  Returns o."""
    L = _ready()
    dims, inputs, dev = _inputs(q, k, v, log_decay)
    p, keep, N = _problem(dims, cu_host, cu_dev, scale, problem_status, scan_segment_chunks, dev)
    slots = state_pool.shape[0]
    pool = _need(state_pool, "state_pool", torch.float32, (slots, dims[3], 128, 128), dev)
    idx = _need(state_indices, "state_indices", torch.int32, (N,), dev)
    resume = _maybe(has_initial_state, "has_initial_state", torch.int32, (N,), dev)
    o = torch.empty_like(v)
    _call(L.gdn_linear_attn_prefill_paged, "gdn_linear_attn_prefill_paged", p, 0,
          (*inputs, pool, slots, idx, resume, o.data_ptr(), _status(device_status, dev)), workspace, dev)
    return o


def linear_attn_bwd(q, k, v, log_decay, d_o, cu_host, cu_dev, scale=None, initial_state=None,
                    d_final_state=None, want_dh0=True, workspace=None, device_status=None,
                    scan_segment_chunks=0):
    """gdn_linear_attn_bwd on torch tensors.  Returns dict dq, dk, dv, dh0."""
    L = _ready()
    dims, inputs, dev = _inputs(q, k, v, log_decay)
    p, keep, N = _problem(dims, cu_host, cu_dev, scale, device_status, scan_segment_chunks, dev)
    shape = (N, dims[3], 128, 128)
    do = _need(d_o, "d_o", torch.bfloat16, v.shape, dev)
    h0 = _maybe(initial_state, "initial_state", torch.float32, shape, dev)
    dht = _maybe(d_final_state, "d_final_state", torch.float32, shape, dev)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dh0 = torch.empty(shape, dtype=torch.float32, device=q.device) if want_dh0 else None
    _call(L.gdn_linear_attn_bwd, "gdn_linear_attn_bwd", p, 1,
          (*inputs, h0, do, dht, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), None if dh0 is None else dh0.data_ptr()),
          workspace, dev)
    return dict(dq=dq, dk=dk, dv=dv, dh0=dh0)


def linear_attn_step(q, k, v, log_decay, state_pool, state_indices, scale=None, device_status=None):
    """gdn_linear_attn_step on torch tensors (state_pool updated in place): row b is one token of
    the sequence in slot state_indices[b].  Returns o."""
    L = _ready()
    (B, H, K, HV, V), (qp, kp, vp, gp), dev = _inputs(q, k, v, log_decay)
    slots = state_pool.shape[0]
    pool = _need(state_pool, "state_pool", torch.float32, (slots, HV, V, K), dev)
    idx = _need(state_indices, "state_indices", torch.int32, (B,), dev)
    o = torch.empty_like(v)
    st = L.gdn_linear_attn_step(B, H, HV, K, V, scale or 0.0, qp, kp, vp, gp, pool, slots, idx, o.data_ptr(),
                                _status(device_status, dev), _raw_stream(dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_linear_attn_step")
    return o


def rope_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, trained_len=0.0, low_turns=1.0,
                     high_turns=32.0, device=None):
    """gdn_rope_frequencies as a tensor [2, rot_dim / 2] (turns per position, head and tail),
    for the `freq` argument of rope; device: where to put it (default: the current CUDA device)."""
    _ready()
    freq = torch.empty((2, rot_dim // 2), dtype=torch.float32)
    st = binding.gdn_rope_frequencies(int(rot_dim), float(base), _ROPE_SCALING[scaling], float(factor),
                                      float(trained_len), float(low_turns), float(high_turns), freq.data_ptr())
    if st != GDN_OK:
        raise GdnError(st, "gdn_rope_frequencies")
    return freq.to("cuda" if device is None else device)


def rope(q, k, positions, freq, layout="half", mscale=1.0, backward=False, inplace=False):
    """gdn_rope on torch tensors: q [T, Hq, D] and k [T, Hk, D] (or None) bf16, positions int32
    [T], freq as rope_frequencies returns it (2 * freq.shape[1] elements of each head turn).
    backward: the gradient (the rotation by the negative angle, the same mscale).  Returns
    (q, k) rotated, new tensors unless inplace.  No gradient is recorded (rotary does that): in
    place, tensors that ask for one are refused."""
    L = _ready()
    bf = torch.bfloat16
    T, Hq, D = q.shape
    pairs = freq.shape[1]
    dev = _device(q)
    qp = qo = _need(q, "q", bf, (T, Hq, D), dev)
    kp = ko = None
    Hk, qt, kt = 0, q, k
    if k is not None:
        Hk = k.shape[1]
        kp = ko = _need(k, "k", bf, (T, Hk, D), dev)
    pos, turns = _need(positions, "positions", torch.int32, (T,), dev), _need(freq, "freq", torch.float32, (2, pairs), dev)
    if inplace:
        if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
            raise ValueError("rope in place has no gradient: use rotary, or no_grad")
    else:
        qt = torch.empty_like(q)
        qo = qt.data_ptr()
        if k is not None:
            kt = torch.empty_like(k)
            ko = kt.data_ptr()
    st = L.gdn_rope(T, Hq, Hk, D, 2 * pairs, _ROPE_LAYOUT[layout], 1 if backward else 0, mscale, qp, kp, pos, turns,
                    qo, ko, _raw_stream(dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_rope")
    if inplace:   # written through their addresses: tell autograd
        for t in (q, k):
            if t is not None and not t.is_inference():
                torch.autograd.graph.increment_version(t)
    return qt, kt
