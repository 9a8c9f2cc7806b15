"""Host side of the short convolution, the selective scan and the norms: the references' gradients against
differences, argument checks that return before any launch, the Python layer's refusals."""
import ctypes
import os
import re
import shutil
import subprocess
import textwrap

import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn
from chunked_gated_delta_06_gb300 import binding, build, linear, mixer

import mixer_reference as ref

FAKE = 0x10000  # never dereferenced: validation fails first
BAD, NOT_BUILT, SMALL = binding.GDN_ERR_INVALID_ARG, binding.GDN_ERR_UNSUPPORTED, binding.GDN_ERR_WORKSPACE_TOO_SMALL
F32, BF16 = binding.GDN_DTYPE_F32, binding.GDN_DTYPE_BF16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.lib()


# ------------------------------------------------------------------------------ references
def _differences(loss, tensors, grads):
    """Central differences of a loss in 64 bits along one random direction of each tensor."""
    rng = torch.Generator().manual_seed(7)
    for name, at in tensors.items():
        step = torch.randn(at.shape, generator=rng, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            ends.append(loss(**{**tensors, name: at + sign * 1e-5 * step}))
        want = (ends[0] - ends[1]) / 2e-5
        got = float((grads[name] * step).sum())
        # the differences are off by 1e-10 of the third derivative and 1e-11 of the loss
        assert abs(got - want) <= 1e-6 * (1.0 + abs(want) + abs(ends[0])), name


def _rand(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape) + len(shape)), dtype=torch.float64)


@pytest.mark.parametrize("W, silu", [(4, True), (2, True), (3, False)])
def test_convolution_gradient_agrees_with_differences(W, silu):
    cu, C = [0, 3, 3, 4, 12], 3
    t = dict(x=_rand(12, C), w=_rand(C, W), bias=_rand(C), h0=_rand(4, C, W - 1))
    dy, dht = _rand(12, C), _rand(4, C, W - 1)

    def loss(x, w, bias, h0):
        (y, _), last, _, _ = ref.conv(x, w, cu, bias, silu, h0)
        return float((y * dy).sum() + (last * dht).sum())
    _, _, g, _ = ref.conv(t["x"], t["w"], cu, t["bias"], silu, t["h0"], dy, dht)
    _differences(loss, t, dict(x=g["dx"], w=g["dw"], bias=g["db"], h0=g["dh0"]))


@pytest.mark.parametrize("gate", [True, False])
def test_scan_gradient_agrees_with_differences(gate):
    cu, C, Ns, G = [0, 3, 3, 9], 4, 8, 2
    t = dict(x=_rand(9, C), dt=_rand(9, C), A_log=0.3 * _rand(C, Ns), B=_rand(9, G, Ns), C=_rand(9, G, Ns) + 1, D=_rand(C),
             bias=_rand(C) - 1, h0=_rand(3, C, Ns), **(dict(z=_rand(9, C) * 2) if gate else {}))
    dy, dht = _rand(9, C), _rand(3, C, Ns)

    def loss(**kw):
        out = ref.scan(cu=cu, **kw)
        return float((out["y"][0] * dy).sum() + (out["ht"][0] * dht).sum())
    g = ref.scan(cu=cu, dy=dy, dht=dht, **t)
    names = dict(x="dx", dt="ddt", A_log="dA_log", B="dB", C="dC", D="dD", bias="ddt_bias", h0="dh0", z="dz")
    _differences(loss, t, {n: g[names[n]][0] for n in t})


@pytest.mark.parametrize("gate, scaled, offset", [("silu", True, 0.0), ("sigmoid", False, 1.0), (None, True, 0.0)])
def test_norm_gradient_agrees_with_differences(gate, scaled, offset):
    t = dict(x=_rand(5, 6), residual=2 * _rand(5, 6), w=_rand(6), **(dict(z=_rand(5, 6) * 2) if gate else {}),
             **(dict(scale=_rand(6)) if scaled else {}))
    dy, dh = _rand(5, 6), _rand(5, 6)
    kw = dict(gate=gate, eps=1e-3, offset=offset)

    def loss(x, residual, w, z=None, scale=None):
        h = residual + (x if scale is None else scale * x)
        return float((ref.norm(h, w, z, **kw)[0] * dy).sum() + (h * dh).sum())
    h = t["residual"] + (t["scale"] * t["x"] if scaled else t["x"])
    g = ref.norm_bwd(h, t["w"], dy, t.get("z"), dh, t.get("scale"), t["x"], **kw)
    names = dict(x="dx", residual="dresidual", w="dweight", z="dz", scale="dscale")
    _differences(loss, t, {n: g[names[n]][0] for n in t})


# ------------------------------------------------------------------------------ the C entry points
def _pack(cu=(0, 5, 9), dev=FAKE, status=None, tokens=None):
    host = np.asarray(cu, np.int32)
    p = binding.GdnPack(len(host) - 1, int(host[-1]) if tokens is None else tokens,
                        host.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), dev, status)
    p.keep = host
    return p


def _shape(channels=64, groups=1, state_dim=16, dtype=BF16, strides=(0, 0, 0, 0, 0), segment=0):
    return binding.GdnScanShape(channels, groups, state_dim, dtype, *strides, segment)


def _distinct(names, size=1 << 24):
    return {n: size * (i + 1) for i, n in enumerate(names)}


class Conv:
    FWD = ["x", "w", "bias", "s0", "y", "s1"]
    PAGED = ["x", "w", "bias", "pool", "idx", "resume", "y", "status"]
    BWD = ["x", "w", "bias", "s0", "dy", "ds1", "dx", "dw", "db", "ds0", "ws"]
    STEP = ["x", "w", "bias", "pool", "idx", "y", "status"]

    def __init__(self, C=64, W=4, act=1, dtype=BF16, stride=None, slots=4):
        self.args, self.stride, self.slots = (C, W, act, dtype), C if stride is None else stride, slots

    def fwd(self, p, x, w, bias, s0, y, s1):
        return binding.lib().gdn_short_conv_fwd(ctypes.byref(p) if p else None, *self.args, x, self.stride, w, bias, s0, y, s1, None)

    def paged(self, p, x, w, bias, pool, idx, resume, y, status):
        return binding.lib().gdn_short_conv_prefill_paged(ctypes.byref(p), *self.args, x, self.stride, w, bias, pool, self.slots,
                                                          idx, resume, y, status, None)

    def bwd(self, p, x, w, bias, s0, dy, ds1, dx, dw, db, ds0, ws, size=1 << 23):
        return binding.lib().gdn_short_conv_bwd(ctypes.byref(p), *self.args, x, self.stride, w, bias, s0, dy, ds1, dx, dw, db,
                                                ds0, ws, size, None)

    def step(self, batch, x, w, bias, pool, idx, y, status):
        return binding.lib().gdn_short_conv_step(batch, *self.args, x, self.stride, w, bias, pool, self.slots, idx, y, status, None)


class Scan:
    INPUTS = ["x", "dt", "A_log", "B", "C", "D", "z", "bias"]
    FWD = INPUTS + ["s0", "y", "s1", "ws"]
    PAGED = INPUTS + ["pool", "idx", "resume", "y", "status", "ws"]
    BWD = INPUTS + ["s0", "dy", "ds1", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "ds0", "ws"]
    STEP = INPUTS + ["pool", "idx", "y", "status"]

    def __init__(self, slots=4, **kw):
        self.s, self.slots = _shape(**kw), slots

    def fwd(self, p, *a, size=1 << 23):
        return binding.lib().gdn_selective_scan_fwd(ctypes.byref(p) if p else None, ctypes.byref(self.s), *a, size, None)

    def paged(self, p, *a, size=1 << 23):
        return binding.lib().gdn_selective_scan_prefill_paged(ctypes.byref(p), ctypes.byref(self.s), *a[:9], self.slots, *a[9:],
                                                              size, None)

    def bwd(self, p, *a, size=1 << 23):
        return binding.lib().gdn_selective_scan_bwd(ctypes.byref(p), ctypes.byref(self.s), *a, size, None)

    def step(self, batch, *a):
        return binding.lib().gdn_selective_scan_step(batch, ctypes.byref(self.s), *a[:9], self.slots, *a[9:], None)


def _forms(op):
    """(name, call of the operands by name, their order) of an operator's entry points."""
    p = _pack()
    for name, first in (("FWD", p), ("PAGED", p), ("BWD", p), ("STEP", 4)):
        call = getattr(op, name.lower())
        yield name, (lambda a, c=call, f=first, n=getattr(op, name): c(f, *(a[k] for k in n))), getattr(op, name)


@pytest.mark.parametrize("kw, status", [
    (dict(C=0), BAD), (dict(W=1), NOT_BUILT), (dict(W=5), NOT_BUILT), (dict(act=2), BAD), (dict(act=-1), BAD),
    (dict(dtype=2), BAD), (dict(stride=63), BAD), (dict(stride=0), BAD)])
def test_convolution_shapes_are_refused(kw, status):
    for name, call, order in _forms(Conv(**kw)):
        assert call(_distinct(order)) == status, name


@pytest.mark.parametrize("kw, status", [
    (dict(channels=0), BAD), (dict(groups=0), BAD), (dict(groups=65), BAD), (dict(groups=3), NOT_BUILT),
    (dict(state_dim=24), NOT_BUILT), (dict(state_dim=64), NOT_BUILT), (dict(dtype=7), BAD), (dict(segment=-2), BAD),
    (dict(strides=(63, 0, 0, 0, 0)), BAD), (dict(strides=(0, 0, 1, 0, 0)), BAD), (dict(strides=(0, 0, 0, 15, 0)), BAD),
    (dict(strides=(0, 0, 0, 0, -16)), BAD)])
def test_scan_shapes_are_refused(kw, status):
    s = _shape(**kw)
    assert binding.lib().gdn_selective_scan_workspace_bytes(ctypes.byref(_pack()), ctypes.byref(s), 1) == 0
    for name, call, order in _forms(Scan(**kw)):
        assert call(_distinct(order)) == status, name


@pytest.mark.parametrize("kw", [dict(cu=(0, 5, 3)), dict(cu=(1, 5)), dict(dev=None), dict(dev=FAKE + 2),
                                dict(status=FAKE + 1), dict(tokens=10), dict(tokens=-1), dict(cu=(0,), tokens=0)])
def test_packs_are_refused(kw):
    p = _pack(**kw)
    assert binding.lib().gdn_short_conv_workspace_bytes(ctypes.byref(p), 64, 4) == 0
    assert binding.lib().gdn_selective_scan_workspace_bytes(ctypes.byref(p), ctypes.byref(_shape()), 0) == 0
    for op in (Conv(), Scan()):
        for form, names in (("fwd", op.FWD), ("paged", op.PAGED), ("bwd", op.BWD)):
            assert getattr(op, form)(p, *_distinct(names).values()) == BAD, form
    assert Conv().fwd(None, *_distinct(Conv.FWD).values()) == BAD
    assert Scan().fwd(None, *_distinct(Scan.FWD).values()) == BAD


# what each entry point cannot do without, and what it may have less than 16-byte aligned
NEEDED = {"conv": {"FWD": "x w y", "PAGED": "x w pool idx y", "BWD": "x w dy dx dw ws", "STEP": "x w pool idx y"},
          "scan": {"FWD": "x dt A_log B C y", "PAGED": "x dt A_log B C pool idx y",
                   "BWD": "x dt A_log B C dy dx ddt dA dB dC dz ws", "STEP": "x dt A_log B C pool idx y"}}
SMALL_ONES = {"x": 2, "dt": 2, "z": 2, "B": 2, "C": 2, "w": 4, "bias": 4, "A_log": 4, "D": 4, "idx": 4, "resume": 4,
              "status": 4, "dw": 4, "db": 4, "dA": 4, "dD": 4, "dbias": 4, "ws": 256}


@pytest.mark.parametrize("op", [Conv(), Scan()], ids=["conv", "scan"])
def test_missing_and_misaligned_buffers_are_refused(op):
    needed = NEEDED["conv" if isinstance(op, Conv) else "scan"]
    for form, call, order in _forms(op):
        at = _distinct(order)
        for name in needed[form].split():
            assert call({**at, name: None}) == BAD, (form, name)
        for name in order:
            assert call({**at, name: at[name] + SMALL_ONES.get(name, 16) // 2}) == BAD, (form, name)
    op.slots = 0
    for form, call, order in _forms(op):
        if form in ("PAGED", "STEP"):
            assert call(_distinct(order)) == BAD
    assert op.step(-1, *_distinct(op.STEP).values()) == BAD
    op.slots = 4
    assert op.step(0, *[None] * len(op.STEP)) == binding.GDN_OK


OUTPUTS = {"FWD": "y s1", "PAGED": "y pool", "BWD": "dx dw db ds0 ddt dA dB dC dD dz dbias", "STEP": "y pool"}


@pytest.mark.parametrize("op", [Conv(), Scan()], ids=["conv", "scan"])
def test_outputs_over_anything_else_are_refused(op):
    # in whole, over the last bytes and over the first ones (all buffers here have 64 bytes at least but
    # for the four bytes of a status word)
    for form, call, order in _forms(op):
        at = _distinct(order)
        for out in OUTPUTS[form].split():
            if out not in at:
                continue
            for other in order:
                if other in (out, "status") or (other == "ws" and form != "BWD"):   # (no part of it is used there)
                    continue
                if other == "idx" or other == "resume" or out in ("dw", "db", "dA", "dD", "dbias"):
                    assert call({**at, out: at[other]}) == BAD, (form, out, other)
                else:
                    for shift in (0, 16, -16):
                        if other == "ws" and shift:
                            continue
                        assert call({**at, out: at[other] + shift}) == BAD, (form, out, other, shift)


def test_workspaces():
    L = binding.lib()
    p, s = _pack((0, 9000)), _shape()
    assert L.gdn_short_conv_workspace_bytes(ctypes.byref(p), 64, 4) >= 64 * 5 * 4
    assert L.gdn_short_conv_workspace_bytes(ctypes.byref(p), 0, 4) == 0
    assert L.gdn_short_conv_workspace_bytes(ctypes.byref(p), 64, 5) == 0
    assert L.gdn_selective_scan_workspace_bytes(ctypes.byref(p), ctypes.byref(s), 2) == 0
    for back in (0, 1):   # never 0 where the arguments are valid
        assert L.gdn_selective_scan_workspace_bytes(ctypes.byref(_pack((0, 0))), ctypes.byref(s), back) > 0
    need = L.gdn_selective_scan_workspace_bytes(ctypes.byref(p), ctypes.byref(s), 1)
    op = Scan()
    a = _distinct(op.BWD, 1 << 28)
    assert op.bwd(p, *a.values(), size=need - 1) == SMALL
    # one long sequence of few channels is split: a forward without a workspace says so
    f = _distinct(op.FWD, 1 << 28)
    assert op.fwd(p, *{**f, "ws": None}.values(), size=0) == SMALL
    assert L.gdn_selective_scan_workspace_bytes(ctypes.byref(p), ctypes.byref(_shape(segment=-1)), 0) == 256
    c = Conv()
    assert c.bwd(_pack(), *_distinct(Conv.BWD).values(), size=255) == SMALL
    assert L.gdn_rms_norm_workspace_bytes(7, 128, BF16, 0) >= 512
    assert L.gdn_rms_norm_workspace_bytes(7, 128, BF16, 1) >= 1024
    for bad in ((-1, 128, BF16, 0), (7, 0, BF16, 0), (7, 8193, BF16, 0), (7, 128, 5, 0)):
        assert L.gdn_rms_norm_workspace_bytes(*bad) == 0


NORM_FWD = ["x", "residual", "scale", "weight", "z", "y", "h"]
NORM_BWD = ["h", "x", "scale", "weight", "z", "dy", "dh", "dx", "dres", "dz", "dw", "ds", "ws"]


def _norm_fwd(rows=4, dim=128, dtype=BF16, res=F32, gate=1, eps=1e-6, offset=0.0, **at):
    a = {**_distinct(NORM_FWD), **at}
    return binding.lib().gdn_rms_norm_fwd(rows, dim, dtype, res, gate, eps, offset, *(a[n] for n in NORM_FWD), None)


def _norm_bwd(rows=4, dim=128, dtype=BF16, res=F32, gate=1, eps=1e-6, offset=0.0, size=1 << 23, **at):
    a = {**_distinct(NORM_BWD), **at}
    return binding.lib().gdn_rms_norm_bwd(rows, dim, dtype, res, gate, eps, offset, *(a[n] for n in NORM_BWD), size, None)


def test_norm_arguments():
    nan, inf = float("nan"), float("inf")
    for call in (_norm_fwd, _norm_bwd):
        for kw in (dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(dtype=2), dict(res=3), dict(gate=3), dict(gate=0),
                   dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(offset=inf), dict(z=None), dict(weight=None),
                   dict(weight=FAKE + 4), dict(scale=FAKE + 4), dict(z=FAKE + 8), dict(res=binding.GDN_NO_RESIDUAL)):
            assert call(**kw) == BAD, (call, kw)
        assert call(dim=8193) == NOT_BUILT and call(dtype=F32, res=BF16) == NOT_BUILT
    for kw in (dict(x=None), dict(y=None), dict(residual=None), dict(h=None), dict(x=FAKE + 8), dict(y=FAKE + 8),
               dict(h=FAKE + 8), dict(residual=FAKE + 8)):
        assert _norm_fwd(**kw) == BAD, kw
    for kw in (dict(h=None), dict(dy=None), dict(dx=None), dict(dz=None), dict(x=None), dict(scale=None), dict(ds=None),
               dict(dw=None), dict(ws=None), dict(ws=FAKE + 16), dict(dx=FAKE + 8), dict(dh=FAKE + 8), dict(dw=FAKE + 2)):
        assert _norm_bwd(**kw) == BAD, kw
    assert _norm_bwd(size=8) == SMALL
    assert _norm_bwd(res=binding.GDN_NO_RESIDUAL, scale=None, x=None, ds=None) == BAD   # with dh and dres all the same
    assert _norm_fwd(rows=0, x=None, y=None, z=None) == binding.GDN_OK
    for call, names, outs in ((_norm_fwd, NORM_FWD, ("y", "h")), (_norm_bwd, NORM_BWD, ("dx", "dres", "dz", "dw", "ds"))):
        at = _distinct(names)
        for out in outs:
            for other in names:
                if other == out:
                    continue
                for shift in (0, 16) if other != "ws" else (0,):
                    assert call(**{out: at[other] + shift}) == BAD, (out, other, shift)


PROGRAM = textwrap.dedent(r"""
    #include <stddef.h>
    #include <stdio.h>
    #include "gdn.h"
    int main(void) {
        printf("%zu %zu %zu %zu %zu ", sizeof(gdn_pack), offsetof(gdn_pack, total_tokens), offsetof(gdn_pack, cu_seqlens_host),
               offsetof(gdn_pack, cu_seqlens_dev), offsetof(gdn_pack, device_status));
        printf("%zu %zu %zu %zu", sizeof(gdn_scan_shape), offsetof(gdn_scan_shape, x_stride), offsetof(gdn_scan_shape, c_stride),
               offsetof(gdn_scan_shape, segment_tokens));
        return gdn_rms_norm_workspace_bytes(4, 128, GDN_DTYPE_BF16, 0) == 0;
    }
""")


def test_structures_are_those_of_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text(PROGRAM)
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", build.INCLUDE, str(src), "-L", build.PKG, "-lgdn",
                    "-Wl,-rpath," + build.PKG, "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    P, S = binding.GdnPack, binding.GdnScanShape
    assert [int(v) for v in out] == [ctypes.sizeof(P), P.total_tokens.offset, P.cu_seqlens_host.offset, P.cu_seqlens_dev.offset,
                                     P.device_status.offset, ctypes.sizeof(S), S.x_stride.offset, S.c_stride.offset,
                                     S.segment_tokens.offset]
    assert len(mixer._PACK.pack(*[0] * 5)) == ctypes.sizeof(P) and len(mixer._SHAPE.pack(*[0] * 10)) == ctypes.sizeof(S)


def test_every_kernel_checks_its_accesses():
    # (in the source: an access outside is not made on purpose on any GPU)
    for name in ("gdn_conv.cu", "gdn_scan.cu", "gdn_scan_bwd.cu", "gdn_norm.cu", "gdn_norm_bwd.cu"):
        text = open(os.path.join(build.CSRC, name)).read()
        for start in re.finditer(r"__global__", text):
            body = text[start.start():text.index("\n}\n", start.start())]
            kernel = re.search(r"\b(k_\w+)\(", body).group(1)
            assert re.search(r"in_range\(|load_vec<|lane\.load\(", body), kernel


# ------------------------------------------------------------------------------ the Python layer
class _Elsewhere:
    """What the calls look at of a CUDA tensor, with a device of its own; nothing is launched."""

    def __init__(self, dtype, shape, device=0):
        self.dtype, self.shape, self.device, self.is_cuda = dtype, torch.Size(shape), device, device >= 0

    def get_device(self):
        return self.device

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


def _calls():
    """Every call's tensors by argument name."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    cu = dict(cu_host=np.array([0, 6], np.int32))
    C, W, Ns = 8, 4, 16
    conv = dict(x=(bf, (6, C)), weight=(f32, (C, W)), bias=(f32, (C,)))
    packed = dict(cu_dev=(i32, (2,)), device_status=(i32, (1,)))
    cs, ss = (bf, (1, C, W - 1)), (f32, (1, C, Ns))
    ws = dict(workspace=(torch.uint8, (64,)))
    yield gdn.short_conv_fwd, dict(conv, **packed, initial_state=cs), cu
    yield gdn.short_conv_bwd, dict(conv, **packed, **ws, dy=(bf, (6, C)), initial_state=cs, d_final_state=cs), cu
    pool = dict(state_indices=(i32, (1,)), has_initial_state=(i32, (1,)), problem_status=(i32, (1,)))
    yield gdn.short_conv_prefill_paged, dict(conv, **packed, **pool, conv_pool=(bf, (3, C, W - 1))), cu
    yield gdn.short_conv_step, dict(conv, conv_pool=(bf, (3, C, W - 1)), state_indices=(i32, (6,)), device_status=(i32, (1,))), {}
    scan = dict(x=(bf, (6, C)), dt=(bf, (6, C)), A_log=(f32, (C, Ns)), B=(bf, (6, 1, Ns)), C=(bf, (6, 1, Ns)), D=(f32, (C,)),
                z=(bf, (6, C)), dt_bias=(f32, (C,)))
    yield gdn.selective_scan_fwd, dict(scan, **packed, **ws, initial_state=ss), cu
    yield gdn.selective_scan_bwd, dict(scan, **packed, **ws, dy=(bf, (6, C)), initial_state=ss, d_final_state=ss), cu
    yield gdn.selective_scan_prefill_paged, dict(scan, **packed, **pool, **ws, state_pool=(f32, (3, C, Ns))), cu
    yield gdn.selective_scan_step, dict(scan, state_pool=(f32, (3, C, Ns)), state_indices=(i32, (6,)), device_status=(i32, (1,))), {}
    row = (bf, (6, C))
    yield gdn.rms_norm_fwd, dict(x=row, weight=(f32, (C,)), z=row, residual=row, scale=(f32, (C,))), {}
    yield gdn.rms_norm_bwd, dict(h=row, weight=(f32, (C,)), dy=row, z=row, dh=row, scale=(f32, (C,)), x=row, **ws), {}


class _Refused(Exception):
    pass


@pytest.fixture
def no_launch(monkeypatch):
    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 64
                raise _Refused(name)
            return call
    mixer._ready()
    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(linear, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(linear, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch, "empty_like", lambda t: t)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: _Elsewhere(torch.float32, a[0] if isinstance(a[0], tuple) else a[:1]))


def test_tensors_of_another_device_type_or_shape_are_refused(no_launch):
    for call, tensors, rest in _calls():
        with pytest.raises(_Refused):   # all on the current device: the call goes through
            call(**{n: _Elsewhere(*x) for n, x in tensors.items()}, **rest)
        for other, (dtype, shape) in tensors.items():
            for device in (1, -1):
                with pytest.raises((ValueError, TypeError), match="device|CUDA"):
                    call(**{n: _Elsewhere(*x, device=device if n == other else 0) for n, x in tensors.items()}, **rest)
            if other in ("workspace", "device_status", "problem_status"):
                continue
            with pytest.raises((ValueError, TypeError)):
                call(**{n: _Elsewhere(torch.float16 if n == other else x[0], x[1]) for n, x in tensors.items()}, **rest)
            wrong = (*shape[:-1], shape[-1] + 1)
            with pytest.raises(ValueError):
                call(**{n: _Elsewhere(x[0], wrong if n == other else x[1]) for n, x in tensors.items()}, **rest)
        with pytest.raises(ValueError, match="device"):   # all of them on one that is not current
            call(**{n: _Elsewhere(*x, device=1) for n, x in tensors.items()}, **rest)


def test_rows_are_taken_as_they_lie():
    mixer._ready()
    wide = torch.zeros(6, 40)
    dev = wide.get_device()
    view = wide[:, 8:24]
    assert mixer._rows(view, "x", torch.float32, (6, 16), dev) == (view.data_ptr(), 40)
    assert mixer._rows(view.unflatten(1, (2, 8)), "B", torch.float32, (6, 2, 8), dev) == (view.data_ptr(), 40)
    assert mixer._rows(view[:1], "x", torch.float32, (1, 16), dev)[1] == 0
    for bad in (wide[:, ::2][:, :16], torch.zeros(16, 6).t(), torch.zeros(1, 16).expand(6, 16)):
        with pytest.raises(ValueError, match="x"):
            mixer._rows(bad, "x", torch.float32, (6, 16), dev)
    from chunked_gated_delta_06_gb300 import autograd
    assert autograd._dense_rows(view) is view
    for other in (wide[:, ::2], torch.zeros(16, 6).t(), torch.zeros(1, 16).expand(6, 16)):
        assert autograd._dense_rows(other).is_contiguous()


def test_arguments_that_do_not_belong_together(no_launch):
    row, w = _Elsewhere(torch.bfloat16, (6, 8)), _Elsewhere(torch.float32, (8,))
    with pytest.raises(ValueError, match="scale"):
        gdn.rms_norm_bwd(row, w, row, scale=w)
    with pytest.raises(ValueError, match="scale"):
        gdn.rms_norm_bwd(row, w, row, x=row)
    with pytest.raises(KeyError):
        gdn.rms_norm_fwd(row, w, z=row, gate="tanh")
    x, weight = _Elsewhere(torch.bfloat16, (6, 8)), _Elsewhere(torch.float32, (8, 4))
    cu, dev = np.array([0, 6], np.int32), _Elsewhere(torch.int32, (2,))
    with pytest.raises(KeyError):
        gdn.short_conv_fwd(x, weight, cu, dev, activation="relu")
    with pytest.raises(ValueError, match="cu_host"):
        gdn.short_conv_fwd(x, weight, np.array([0, 5], np.int32), dev)
    for W in (0, 1, 5):
        with pytest.raises(ValueError, match="width"):
            gdn.short_conv_fwd(x, _Elsewhere(torch.float32, (8, W)), cu, dev)


@pytest.mark.parametrize("which", ["short_conv", "selective_scan", "rms_norm"])
def test_second_derivatives_that_do_not_exist_are_refused(monkeypatch, which):
    # the gradients of a fused backward are not differentiable: a loss on them must not lose its term
    x, w = torch.randn(4, 8, requires_grad=True), torch.ones(8, 4)
    if which == "short_conv":
        monkeypatch.setattr(mixer, "short_conv_fwd", lambda x, *a, **kw: (x * 2.0, None))
        monkeypatch.setattr(mixer, "short_conv_bwd", lambda x, *a, **kw: dict(dx=x * 0, dw=w * 0, dbias=None, dh0=None))
        y, _ = gdn.short_conv(x, w, cu_seqlens=torch.tensor([0, 4]))
    elif which == "selective_scan":
        B = torch.ones(4, 1, 8)
        names = ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
        monkeypatch.setattr(mixer, "selective_scan_fwd", lambda x, *a, **kw: (x * 2.0, None))
        monkeypatch.setattr(mixer, "selective_scan_bwd", lambda x, *a, **kw: dict(dict.fromkeys(names), dx=x * 0))
        y, _ = gdn.selective_scan(x, x.detach(), w, B, B, cu_seqlens=torch.tensor([0, 4]))
    else:
        monkeypatch.setattr(mixer, "rms_norm_fwd", lambda x, *a, **kw: (x * 2.0, None))
        monkeypatch.setattr(mixer, "rms_norm_bwd", lambda h, *a, **kw: dict(dx=h * 0, dresidual=None, dz=None,
                                                                            dweight=torch.zeros(8), dscale=None))
        y = gdn.rms_norm(x, torch.ones(8))
    (dx,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once more"):
        (dx.square().sum() + y.sum()).backward()


def test_offsets_changed_before_the_backward(monkeypatch):
    # a loop that reuses its offset buffers: the backward has the forward's host copy, and a device
    # copy that changed in place is an error
    seen = []
    monkeypatch.setattr(mixer, "short_conv_fwd", lambda x, *a, **kw: (x * 2.0, None))
    monkeypatch.setattr(mixer, "short_conv_bwd", lambda x, w, dy, cu, cu_dev, **kw: (
        seen.append(cu.copy()), dict(dx=x * 0, dw=w * 0, dbias=None, dh0=None))[1])
    x, w = torch.randn(4, 8, requires_grad=True), torch.ones(8, 4)
    host, dev = torch.tensor([0, 1, 4], dtype=torch.int32), torch.tensor([0, 1, 4], dtype=torch.int32)
    y, _ = gdn.short_conv(x, w, cu_seqlens=dev, cu_seqlens_cpu=host)
    host[1] = 3
    y.sum().backward()
    assert seen[0].tolist() == [0, 1, 4]
    y, _ = gdn.short_conv(x, w, cu_seqlens=dev, cu_seqlens_cpu=host)
    dev[1] = 3
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_channels_that_indices_do_not_hold_are_refused(lib):
    most = 1 << 30
    p = _pack()
    assert lib.gdn_short_conv_workspace_bytes(ctypes.byref(p), most, 4) > 0
    assert lib.gdn_short_conv_workspace_bytes(ctypes.byref(p), most + 1, 4) == 0
    assert lib.gdn_selective_scan_workspace_bytes(ctypes.byref(p), ctypes.byref(_shape(most)), 0) > 0
    assert lib.gdn_selective_scan_workspace_bytes(ctypes.byref(p), ctypes.byref(_shape(most + 1)), 0) == 0
    assert lib.gdn_short_conv_step(1, most + 1, 4, 0, BF16, FAKE, most + 1, FAKE, None, 2 * FAKE, 2, 4, 3 * FAKE, None, None) == BAD
    assert lib.gdn_selective_scan_step(1, ctypes.byref(_shape(most + 1)), *[FAKE] * 5, None, None, None, FAKE, 2, FAKE, FAKE,
                                       None, None) == BAD


def test_parts_of_tensors_become_whole_ones():
    own = gdn.autograd._aligned
    wide = torch.arange(64, dtype=torch.float32)
    assert wide.data_ptr() % 16 == 0 and own(wide) is wide and own(None) is None
    assert own(wide[4:]).data_ptr() == wide[4:].data_ptr()
    part = own(wide[1:9])
    assert part.data_ptr() % 16 == 0 and torch.equal(part, wide[1:9])
    turned = own(wide.view(8, 8).t())
    assert turned.is_contiguous() and torch.equal(turned, wide.view(8, 8).t())
