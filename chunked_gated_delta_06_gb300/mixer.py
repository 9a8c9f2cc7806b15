"""The short causal convolution, the selective state space scan and the norms with their gate and
residual on torch tensors: argument checks and marshalling only, every step of the computation runs
in libgdn's CUDA kernels.

Activations are bf16 or fp32 (all tensors of a call alike); parameters are fp32.  Rows of an input
[T, ...] may lie apart (a slice of a wider projection): the elements of a row must be dense.  Other
tensors are dense and start on 16 bytes, as a new tensor does and a part of one may not.
"""
from __future__ import annotations

import numpy as np

from . import binding, linear
from .binding import (GDN_ACT_NONE, GDN_ACT_SILU, GDN_DTYPE_BF16, GDN_DTYPE_F32, GDN_ERR_WORKSPACE_TOO_SMALL,
                      GDN_GATE_NONE, GDN_GATE_SIGMOID, GDN_GATE_SILU, GDN_NO_RESIDUAL, GDN_OK, GdnError)
from .linear import _maybe, _need, _status, _struct_of

_PACK = _struct_of(binding.GdnPack)
_SHAPE = _struct_of(binding.GdnScanShape)
_ACTIVATION = {None: GDN_ACT_NONE, "none": GDN_ACT_NONE, "silu": GDN_ACT_SILU}
_GATE = {None: GDN_GATE_NONE, "none": GDN_GATE_NONE, "silu": GDN_GATE_SILU, "sigmoid": GDN_GATE_SIGMOID}

torch = None
_DTYPE = {}


def _ready():
    global torch
    L = linear._ready()
    if torch is None:
        torch = linear.torch
        _DTYPE.update({torch.bfloat16: GDN_DTYPE_BF16, torch.float32: GDN_DTYPE_F32})
    return L


def _first(t, name):
    """The device and the type of a call, from its first tensor."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dev != linear._current_device():
        raise ValueError("%s is on cuda:%d, which is not the current device" % (name, dev))
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError("%s must be bfloat16 or float32, not %s" % (name, t.dtype))
    return dev, code


def _rows(t, name, dtype, shape, dev):
    """Address and row distance of a tensor whose rows are dense."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or t.is_contiguous():
        at = _need(t, name, dtype, shape, dev)
        return at, 0
    width, stride = 1, t.stride()
    for n, s in zip(reversed(shape[1:]), reversed(stride[1:])):
        if n != 1 and s != width:
            raise ValueError("%s must have dense rows" % name)
        width *= n
    if shape[0] > 1 and stride[0] < width:
        raise ValueError("%s has rows that overlap" % name)
    return t.data_ptr(), stride[0] if shape[0] > 1 else 0


def _int32(sizes):
    """Refuse sizes that the library's 32-bit arguments would wrap.  sizes: their bits, or-ed."""
    if sizes >> 31:
        raise ValueError("the sizes of a call must be below 2^31")


def _pack(T, cu_host, cu_dev, status, dev):
    """gdn_pack as bytes, the array that it points at (to be kept alive), and N."""
    cu = cu_host
    if type(cu) is not np.ndarray or cu.dtype != np.int32 or not cu.flags.c_contiguous:
        cu = np.ascontiguousarray(np.asarray(cu_host, dtype=np.int32))
    N = len(cu) - 1
    if N < 1 or cu[N] != T:
        raise ValueError("cu_host must end with the number of tokens, %d" % T)
    # (in the order of GdnPack)
    return _PACK.pack(N, T, cu.__array_interface__["data"][0], _need(cu_dev, "cu_dev", torch.int32, (N + 1,), dev),
                      _status(status, dev) or 0), cu, N


def _scratch(workspace, need, dev):
    """Address and bytes of a call's workspace: the caller's, or a new one."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the call's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _done(status, name):
    if status != GDN_OK:
        raise GdnError(status, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------------------ convolution
def _conv(x, weight, bias):
    if x.dim() != 2 or weight.dim() != 2 or not 2 <= weight.shape[1] <= 4:
        raise ValueError("x must be [tokens, channels] and weight [channels, width], width 2, 3 or 4")
    dev, code = _first(x, "x")
    T, C = x.shape
    W = weight.shape[1]
    _int32(T | C)
    xp, stride = _rows(x, "x", x.dtype, (T, C), dev)
    f32 = torch.float32
    return (T, C, W), dev, code, (xp, stride or C, _need(weight, "weight", f32, (C, W), dev),
                                  _maybe(bias, "bias", f32, (C,), dev))


def short_conv_fwd(x, weight, cu_host, cu_dev, bias=None, activation="silu", initial_state=None,
                   output_final_state=True, device_status=None):
    """gdn_short_conv_fwd on torch tensors.  Returns (y, final_state or None).

    x: [T, C], bf16 or fp32; weight: fp32 [C, W], W = 2, 3 or 4; bias: fp32 [C]; activation: "silu" or
    None; states [N, C, W - 1] in x's type: the last inputs, oldest first."""
    L = _ready()
    (T, C, W), dev, code, args = _conv(x, weight, bias)
    p, keep, N = _pack(T, cu_host, cu_dev, device_status, dev)
    h0 = _maybe(initial_state, "initial_state", x.dtype, (N, C, W - 1), dev)
    y = torch.empty((T, C), dtype=x.dtype, device=x.device)
    ht = torch.empty((N, C, W - 1), dtype=x.dtype, device=x.device) if output_final_state else None
    _done(L.gdn_short_conv_fwd(p, C, W, _ACTIVATION[activation], code, *args, h0, y.data_ptr(), _ptr(ht),
                               linear._raw_stream(dev)), "gdn_short_conv_fwd")
    return y, ht


def short_conv_prefill_paged(x, weight, cu_host, cu_dev, conv_pool, state_indices, has_initial_state=None, bias=None,
                             activation="silu", device_status=None, problem_status=None):
    """gdn_short_conv_prefill_paged on torch tensors (conv_pool [slots, C, W - 1] updated in place; slots
    and status words as in chunk_prefill_paged).  Returns y."""
    L = _ready()
    (T, C, W), dev, code, args = _conv(x, weight, bias)
    p, keep, N = _pack(T, cu_host, cu_dev, problem_status, dev)
    slots = conv_pool.shape[0]
    _int32(slots)
    pool = _need(conv_pool, "conv_pool", x.dtype, (slots, C, W - 1), dev)
    idx = _need(state_indices, "state_indices", torch.int32, (N,), dev)
    resume = _maybe(has_initial_state, "has_initial_state", torch.int32, (N,), dev)
    y = torch.empty((T, C), dtype=x.dtype, device=x.device)
    _done(L.gdn_short_conv_prefill_paged(p, C, W, _ACTIVATION[activation], code, *args, pool, slots, idx, resume,
                                         y.data_ptr(), _status(device_status, dev), linear._raw_stream(dev)),
          "gdn_short_conv_prefill_paged")
    return y


def short_conv_bwd(x, weight, dy, cu_host, cu_dev, bias=None, activation="silu", initial_state=None,
                   d_final_state=None, want_dh0=True, workspace=None, device_status=None):
    """gdn_short_conv_bwd on torch tensors.  Returns dict dx, dw, dbias, dh0 (dbias None without a bias)."""
    L = _ready()
    (T, C, W), dev, code, args = _conv(x, weight, bias)
    p, keep, N = _pack(T, cu_host, cu_dev, device_status, dev)
    state = (N, C, W - 1)
    do = _need(dy, "dy", x.dtype, (T, C), dev)
    h0 = _maybe(initial_state, "initial_state", x.dtype, state, dev)
    dht = _maybe(d_final_state, "d_final_state", x.dtype, state, dev)
    dx = torch.empty((T, C), dtype=x.dtype, device=x.device)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dh0 = torch.empty(state, dtype=x.dtype, device=x.device) if want_dh0 else None
    ws, n, keep_ws = _scratch(workspace, L.gdn_short_conv_workspace_bytes(p, C, W), dev)
    _done(L.gdn_short_conv_bwd(p, C, W, _ACTIVATION[activation], code, *args, h0, do, dht, dx.data_ptr(), dw.data_ptr(),
                               _ptr(db), _ptr(dh0), ws, n, linear._raw_stream(dev)), "gdn_short_conv_bwd")
    return dict(dx=dx, dw=dw, dbias=db, dh0=dh0)


def short_conv_step(x, weight, conv_pool, state_indices, bias=None, activation="silu", device_status=None):
    """gdn_short_conv_step on torch tensors (conv_pool updated in place): row b of x [B, C] is one token of
    the sequence in slot state_indices[b].  Returns y."""
    L = _ready()
    (B, C, W), dev, code, args = _conv(x, weight, bias)
    slots = conv_pool.shape[0]
    _int32(slots)
    pool = _need(conv_pool, "conv_pool", x.dtype, (slots, C, W - 1), dev)
    idx = _need(state_indices, "state_indices", torch.int32, (B,), dev)
    y = torch.empty((B, C), dtype=x.dtype, device=x.device)
    _done(L.gdn_short_conv_step(B, C, W, _ACTIVATION[activation], code, *args, pool, slots, idx, y.data_ptr(),
                                _status(device_status, dev), linear._raw_stream(dev)), "gdn_short_conv_step")
    return y


# ------------------------------------------------------------------------------ scan
def _scan(x, dt, A_log, B, C, D, z, dt_bias, segment_tokens):
    """Sizes, device, gdn_scan_shape as bytes and the addresses from x to dt_bias."""
    if x.dim() != 2 or B.dim() != 3:
        raise ValueError("x must be [tokens, channels], B and C [tokens, groups, state_dim]")
    dev, code = _first(x, "x")
    T, Ch = x.shape
    _, G, Ns = B.shape
    _int32(T | Ch | G | Ns)
    t, f32 = x.dtype, torch.float32
    xp, xs = _rows(x, "x", t, (T, Ch), dev)
    dp, ds = _rows(dt, "dt", t, (T, Ch), dev)
    bp, bs = _rows(B, "B", t, (T, G, Ns), dev)
    cp, cs = _rows(C, "C", t, (T, G, Ns), dev)
    zp, zs = (None, 0) if z is None else _rows(z, "z", t, (T, Ch), dev)
    # (in the order of GdnScanShape)
    shape = _SHAPE.pack(Ch, G, Ns, code, xs, ds, zs, bs, cs, segment_tokens)
    return (T, Ch, G, Ns), dev, shape, (xp, dp, _need(A_log, "A_log", f32, (Ch, Ns), dev), bp, cp,
                                        _maybe(D, "D", f32, (Ch,), dev), zp, _maybe(dt_bias, "dt_bias", f32, (Ch,), dev))


def _scan_call(fn, name, p, shape, T, args, workspace, dev):
    """With a workspace of the caller's or a new one; up to 64 tokens, which the library's plan does not
    split, first without."""
    stream = linear._raw_stream(dev)
    ws, n = None, 0
    if workspace is not None:
        ws, n, keep = _scratch(workspace, 0, dev)
    elif T > 64:
        ws, n, keep = _scratch(None, binding._lib.gdn_selective_scan_workspace_bytes(p, shape, 0), dev)
    st = fn(p, shape, *args, ws, n, stream)
    if st == GDN_ERR_WORKSPACE_TOO_SMALL and ws is None:   # (segments that the caller asked for)
        ws, n, keep = _scratch(None, binding._lib.gdn_selective_scan_workspace_bytes(p, shape, 0), dev)
        st = fn(p, shape, *args, ws, n, stream)
    _done(st, name)


def selective_scan_fwd(x, dt, A_log, B, C, cu_host, cu_dev, D=None, z=None, dt_bias=None, initial_state=None,
                       output_final_state=True, workspace=None, device_status=None, segment_tokens=0):
    """gdn_selective_scan_fwd on torch tensors.  Returns (y, final_state or None).

    x, dt, z: [T, channels]; B, C: [T, groups, state_dim], all bf16 or all fp32; A_log: fp32 [channels,
    state_dim], state_dim = 8, 16 or 32; D, dt_bias: fp32 [channels]; states fp32 [N, channels, state_dim].
    segment_tokens: 0 = the library's plan, -1 = never split, L > 0 = segments of L tokens."""
    L = _ready()
    (T, Ch, G, Ns), dev, shape, inputs = _scan(x, dt, A_log, B, C, D, z, dt_bias, segment_tokens)
    p, keep, N = _pack(T, cu_host, cu_dev, device_status, dev)
    state = (N, Ch, Ns)
    h0 = _maybe(initial_state, "initial_state", torch.float32, state, dev)
    y = torch.empty((T, Ch), dtype=x.dtype, device=x.device)
    ht = torch.empty(state, dtype=torch.float32, device=x.device) if output_final_state else None
    _scan_call(L.gdn_selective_scan_fwd, "gdn_selective_scan_fwd", p, shape, T,
               (*inputs, h0, y.data_ptr(), _ptr(ht)), workspace, dev)
    return y, ht


def selective_scan_prefill_paged(x, dt, A_log, B, C, cu_host, cu_dev, state_pool, state_indices,
                                 has_initial_state=None, D=None, z=None, dt_bias=None, device_status=None,
                                 workspace=None, problem_status=None, segment_tokens=0):
    """gdn_selective_scan_prefill_paged on torch tensors (state_pool fp32 [slots, channels, state_dim] updated
    in place; slots and status words as in chunk_prefill_paged).  Returns y."""
    L = _ready()
    (T, Ch, G, Ns), dev, shape, inputs = _scan(x, dt, A_log, B, C, D, z, dt_bias, segment_tokens)
    p, keep, N = _pack(T, cu_host, cu_dev, problem_status, dev)
    slots = state_pool.shape[0]
    _int32(slots)
    pool = _need(state_pool, "state_pool", torch.float32, (slots, Ch, Ns), dev)
    idx = _need(state_indices, "state_indices", torch.int32, (N,), dev)
    resume = _maybe(has_initial_state, "has_initial_state", torch.int32, (N,), dev)
    y = torch.empty((T, Ch), dtype=x.dtype, device=x.device)
    _scan_call(L.gdn_selective_scan_prefill_paged, "gdn_selective_scan_prefill_paged", p, shape, T,
               (*inputs, pool, slots, idx, resume, y.data_ptr(), _status(device_status, dev)), workspace, dev)
    return y


def selective_scan_bwd(x, dt, A_log, B, C, dy, cu_host, cu_dev, D=None, z=None, dt_bias=None, initial_state=None,
                       d_final_state=None, want_dh0=True, workspace=None, device_status=None, segment_tokens=0):
    """gdn_selective_scan_bwd on torch tensors.  Returns dict dx, ddt, dA_log, dB, dC, dD, dz, ddt_bias, dh0
    (None for what the call has no input of)."""
    L = _ready()
    (T, Ch, G, Ns), dev, shape, inputs = _scan(x, dt, A_log, B, C, D, z, dt_bias, segment_tokens)
    p, keep, N = _pack(T, cu_host, cu_dev, device_status, dev)
    state, t, f32 = (N, Ch, Ns), x.dtype, torch.float32
    do = _need(dy, "dy", t, (T, Ch), dev)
    h0 = _maybe(initial_state, "initial_state", f32, state, dev)
    dht = _maybe(d_final_state, "d_final_state", f32, state, dev)
    new = lambda size, kind, there=True: torch.empty(size, dtype=kind, device=x.device) if there else None  # noqa: E731
    out = dict(dx=new((T, Ch), t), ddt=new((T, Ch), t), dA_log=new((Ch, Ns), f32), dB=new((T, G, Ns), t),
               dC=new((T, G, Ns), t), dD=new((Ch,), f32, D is not None), dz=new((T, Ch), t, z is not None),
               ddt_bias=new((Ch,), f32, dt_bias is not None), dh0=new(state, f32, want_dh0))
    ws, n, keep_ws = _scratch(workspace, L.gdn_selective_scan_workspace_bytes(p, shape, 1), dev)
    _done(L.gdn_selective_scan_bwd(p, shape, *inputs, h0, do, dht, *map(_ptr, out.values()), ws, n,
                                   linear._raw_stream(dev)), "gdn_selective_scan_bwd")
    return out


def selective_scan_step(x, dt, A_log, B, C, state_pool, state_indices, D=None, z=None, dt_bias=None,
                        device_status=None):
    """gdn_selective_scan_step on torch tensors (state_pool updated in place): row b is one token of the
    sequence in slot state_indices[b].  Returns y."""
    L = _ready()
    (rows, Ch, G, Ns), dev, shape, inputs = _scan(x, dt, A_log, B, C, D, z, dt_bias, 0)
    slots = state_pool.shape[0]
    _int32(slots)
    pool = _need(state_pool, "state_pool", torch.float32, (slots, Ch, Ns), dev)
    idx = _need(state_indices, "state_indices", torch.int32, (rows,), dev)
    y = torch.empty((rows, Ch), dtype=x.dtype, device=x.device)
    _done(L.gdn_selective_scan_step(rows, shape, *inputs, pool, slots, idx, y.data_ptr(), _status(device_status, dev),
                                    linear._raw_stream(dev)), "gdn_selective_scan_step")
    return y


# ------------------------------------------------------------------------------ norm
def rms_norm_fwd(x, weight, z=None, residual=None, scale=None, gate="silu", eps=1e-6, offset=0.0):
    """gdn_rms_norm_fwd on torch tensors.  Returns (y, h): h = residual + scale x in residual's type (None
    without a residual), y = h / rms(h) (offset + weight) act(z) in x's.

    x, z, residual: [..., dim], bf16 or fp32 (a bf16 x may have an fp32 residual); weight, scale: fp32 [dim];
    gate: "silu" or "sigmoid", of z (without z it is not looked at)."""
    L = _ready()
    dev, code = _first(x, "x")
    shape, D, t = x.shape, x.shape[-1], x.dtype
    rows = x.numel() // D if D else 0
    _int32(D)
    kind = GDN_NO_RESIDUAL if residual is None else _first(residual, "residual")[1]
    f32 = torch.float32
    args = (_need(x, "x", t, shape, dev), None if residual is None else _need(residual, "residual", residual.dtype, shape, dev),
            _maybe(scale, "scale", f32, (D,), dev), _need(weight, "weight", f32, (D,), dev), _maybe(z, "z", t, shape, dev))
    y = torch.empty_like(x)
    h = None if residual is None else torch.empty_like(residual)
    _done(L.gdn_rms_norm_fwd(rows, D, code, kind, GDN_GATE_NONE if z is None else _GATE[gate], eps, offset, *args,
                             y.data_ptr(), _ptr(h), linear._raw_stream(dev)), "gdn_rms_norm_fwd")
    return y, h


def rms_norm_bwd(h, weight, dy, z=None, dh=None, scale=None, x=None, gate="silu", eps=1e-6, offset=0.0,
                 residual=False, workspace=None):
    """gdn_rms_norm_bwd on torch tensors.  Returns dict dx, dresidual, dz, dweight, dscale (None for what the
    call has no input of).

    h: the forward's h, or its x where there was no residual; x: the forward's x, with a scale only; dh:
    the gradient of h.  There was a residual where dh or a scale is given, h and dy have two types, or
    `residual` says so; without a scale and in one type dresidual is dx itself, the same tensor."""
    L = _ready()
    dev, code = _first(dy, "dy")
    shape, D, t = dy.shape, dy.shape[-1], dy.dtype
    rows = dy.numel() // D if D else 0
    _int32(D)
    there = residual or dh is not None or scale is not None or h.dtype is not t
    if (scale is None) != (x is None):
        raise ValueError("x is given with a scale, and only then")
    kind = _first(h, "h")[1] if there else GDN_NO_RESIDUAL
    f32, r = torch.float32, h.dtype
    args = (_need(h, "h", r, shape, dev), _maybe(x, "x", t, shape, dev), _maybe(scale, "scale", f32, (D,), dev),
            _need(weight, "weight", f32, (D,), dev), _maybe(z, "z", t, shape, dev), _need(dy, "dy", t, shape, dev),
            _maybe(dh, "dh", r, shape, dev))
    dx = torch.empty_like(dy)
    dres = dx if there else None
    if there and (scale is not None or r is not t):
        dres = torch.empty_like(h)
    dz = None if z is None else torch.empty_like(z)
    dw = torch.empty_like(weight)
    ds = None if scale is None else torch.empty_like(scale)
    ws, n, keep = _scratch(workspace, L.gdn_rms_norm_workspace_bytes(rows, D, code, scale is not None), dev)
    _done(L.gdn_rms_norm_bwd(rows, D, code, kind, GDN_GATE_NONE if z is None else _GATE[gate], eps, offset, *args,
                             dx.data_ptr(), None if dres is dx else _ptr(dres), _ptr(dz), dw.data_ptr(), _ptr(ds), ws, n,
                             linear._raw_stream(dev)), "gdn_rms_norm_bwd")
    return dict(dx=dx, dresidual=dres, dz=dz, dweight=dw, dscale=ds)
