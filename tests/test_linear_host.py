"""Host side of the decay-only linear attention and of rotary positions: the references'
gradients against differences, argument checks that return before any launch, frequencies."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn
from chunked_gated_delta_06_gb300 import binding, build, linear

import linear_reference as ref

FAKE = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.lib()


def _problem(cu, H=2, HV=4, K=128, V=128, dev=0x1000):
    return binding.make_problem(cu, H, HV, K, V, 0.0, cu_dev_ptr=dev)


def test_reference_gradients_agree_with_differences():
    rng = np.random.default_rng(5)
    cu, H, HV = [0, 3, 3, 8], 1, 2
    T = cu[-1]
    x = dict(q=rng.standard_normal((T, H, 128)), k=rng.standard_normal((T, H, 128)),
             v=rng.standard_normal((T, HV, 128)), h0=rng.standard_normal((3, HV, 128, 128)))
    g = np.array([-0.3, 0.0])
    do, dht = rng.standard_normal((T, HV, 128)), rng.standard_normal((3, HV, 128, 128))

    def loss(d):
        o, fin = ref.forward(d["q"], d["k"], d["v"], g, cu, d["h0"])
        return float((o * do).sum() + (fin * dht).sum())
    gr = ref.backward(x["q"], x["k"], x["v"], g, cu, do, x["h0"], dht)
    for name, got in (("q", gr["dq"]), ("k", gr["dk"]), ("v", gr["dv"]), ("h0", gr["dh0"])):
        step = rng.standard_normal(x[name].shape)
        eps = 1e-5
        up, dn = dict(x), dict(x)
        up[name], dn[name] = x[name] + eps * step, x[name] - eps * step
        want = (loss(up) - loss(dn)) / (2 * eps)
        # the loss is at most bilinear in any one input: central differences are exact but for
        # rounding, about 1e-16 * |loss| / eps
        assert abs((got * step).sum() - want) <= 1e-6 * (1.0 + abs(want)), name


@pytest.mark.parametrize("mut, status", [
    (dict(K=64), binding.GDN_ERR_UNSUPPORTED),
    (dict(H=3, HV=4), binding.GDN_ERR_UNSUPPORTED),
    (dict(cu=[0, 5, 3]), binding.GDN_ERR_INVALID_ARG),
    (dict(dev=0), binding.GDN_ERR_INVALID_ARG),
])
def test_invalid_problems_are_refused(mut, status):
    kw = dict(cu=[0, 5, 9])
    kw.update(mut)
    p, keep = _problem(**kw)
    assert gdn.gdn_linear_attn_workspace_bytes(p, 0) == 0
    assert gdn.gdn_linear_attn_fwd(p, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, 1 << 40, None) == status
    assert gdn.gdn_linear_attn_bwd(p, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, None,
                                   FAKE, 1 << 40, None) == status
    assert gdn.gdn_linear_attn_prefill_paged(p, FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, None, FAKE, None,
                                             FAKE, 1 << 40, None) == status


def test_missing_and_misaligned_buffers_are_refused():
    p, keep = _problem([0, 5, 9])
    bad = binding.GDN_ERR_INVALID_ARG
    fwd = [FAKE] * 4 + [None, FAKE, None, FAKE, 1 << 40, None]
    for i, x in ((0, None), (1, None), (2, None), (3, None), (5, None), (7, None),
                 (0, FAKE + 2), (3, FAKE + 2), (4, FAKE + 4), (7, FAKE + 16)):
        a = list(fwd)
        a[i] = x
        assert gdn.gdn_linear_attn_fwd(p, *a) == bad, i
    a = list(fwd)
    a[4] = a[6] = FAKE  # the final state over the initial state
    assert gdn.gdn_linear_attn_fwd(p, *a) == bad
    a = list(fwd)
    a[8] = 0
    assert gdn.gdn_linear_attn_fwd(p, *a) == binding.GDN_ERR_WORKSPACE_TOO_SMALL
    bwd = [FAKE] * 4 + [None, FAKE, None, FAKE, FAKE, FAKE, None, FAKE, 1 << 40, None]
    for i, x in ((3, None), (5, None), (7, None), (8, None), (9, None), (11, None), (5, FAKE + 8)):
        a = list(bwd)
        a[i] = x
        assert gdn.gdn_linear_attn_bwd(p, *a) == bad, i
    a = list(bwd)
    a[12] = gdn.gdn_linear_attn_workspace_bytes(p, 1) - 1
    assert gdn.gdn_linear_attn_bwd(p, *a) == binding.GDN_ERR_WORKSPACE_TOO_SMALL
    paged = [FAKE] * 5 + [4, FAKE, None, FAKE, None, FAKE, 1 << 40, None]
    for i, x in ((4, None), (5, 0), (6, None), (4, FAKE + 4), (9, FAKE + 2)):
        a = list(paged)
        a[i] = x
        assert gdn.gdn_linear_attn_prefill_paged(p, *a) == bad, i
    assert gdn.gdn_linear_attn_workspace_bytes(p, 2) == 0
    assert gdn.gdn_linear_attn_workspace_bytes(p, -1) == 0
    assert gdn.gdn_linear_attn_workspace_bytes(p, 0) > 0 and gdn.gdn_linear_attn_workspace_bytes(p, 1) > 0


def test_backward_outputs_over_inputs_are_refused():
    # dq, dk, dv and dh0 are written while the other scans still read: no overlap, in whole or part
    p, keep = _problem([0, 5, 9])
    names = ["q", "k", "v", "g", "h0", "do", "dht", "dq", "dk", "dv", "dh0", "ws"]
    at = {n: 0x10000000 * (i + 1) for i, n in enumerate(names)}
    tokens = dict(q=2, k=2, v=4, do=4, dq=2, dk=2, dv=4)
    size = {n: 9 * tokens[n] * 256 if n in tokens else 2 * 4 * 65536 for n in names}
    size["g"] = 16
    for out in ("dq", "dk", "dv", "dh0"):
        for other in names:
            if other in (out, "ws"):
                continue
            for place in (at[other], at[other] + (size[other] - 16 if other != "g" else 0),
                          at[other] - size[out] + 16):
                a = dict(at)
                a[out] = place
                got = gdn.gdn_linear_attn_bwd(p, *(a[n] for n in names), 1 << 20, None)
                assert got == binding.GDN_ERR_INVALID_ARG, (out, other, hex(place))


@pytest.mark.parametrize("H", [2, 4])
def test_forward_outputs_over_inputs_are_refused(H):
    # o, the final state and the pool over anything else in part, or over a tensor of another shape:
    # value heads and sequences are walked at once.  (o as one of q, k, v itself is read before it is written.)
    p, keep = _problem([0, 5, 9], H=H)
    fwd = ["q", "k", "v", "g", "h0", "o", "ht", "ws"]
    paged = ["q", "k", "v", "g", "pool", "idx", "resume", "o", "status", "ws"]
    heads = dict(q=H, k=H, v=4, o=4)
    size = {n: 9 * heads[n] * 256 if n in heads else 2 * 4 * 65536 for n in fwd}
    size.update(g=16, pool=3 * 4 * 65536, idx=8, resume=8, status=4)
    for names, outs in ((fwd, ("o", "ht")), (paged, ("o", "pool"))):
        at = {n: 0x10000000 * (i + 1) for i, n in enumerate(names)}
        for out in outs:
            for other in names:
                if other in (out, "ws"):
                    continue
                for shift in (0, (size[other] - 1) // 16 * 16, 16 - size[out]):
                    if shift == 0 and out == "o" and other in heads and size[other] == size["o"]:
                        continue
                    a = dict(at)
                    a[out] = at[other] + shift
                    if names is fwd:
                        got = gdn.gdn_linear_attn_fwd(p, *(a[n] for n in names), 1 << 20, None)
                    else:
                        args = [a[n] for n in names]
                        got = gdn.gdn_linear_attn_prefill_paged(p, *args[:5], 3, *args[5:], 1 << 20, None)
                    assert got == binding.GDN_ERR_INVALID_ARG, (out, other, shift)


def test_step_arguments():
    def call(batch=4, H=2, HV=4, K=128, pool=FAKE, slots=8, idx=FAKE, g=FAKE, q=FAKE):
        return gdn.gdn_linear_attn_step(batch, H, HV, K, 128, 0.0, q, FAKE, FAKE, g, pool, slots, idx, FAKE,
                                        None, None)
    assert call(K=64) == binding.GDN_ERR_UNSUPPORTED
    assert call(H=3) == binding.GDN_ERR_UNSUPPORTED
    for kw in (dict(batch=-1), dict(slots=0), dict(idx=None), dict(pool=FAKE + 4), dict(g=None),
               dict(g=FAKE + 2), dict(q=FAKE + 4)):
        assert call(**kw) == binding.GDN_ERR_INVALID_ARG, kw
    assert call(batch=0) == binding.GDN_OK


def test_rope_arguments():
    def call(T=4, Hq=2, Hk=1, D=128, rot=64, layout=0, backward=0, m=1.0, q=FAKE, k=FAKE, pos=FAKE,
             freq=FAKE, qo=FAKE, ko=FAKE):
        return gdn.gdn_rope(T, Hq, Hk, D, rot, layout, backward, m, q, k, pos, freq, qo, ko, None)
    for kw in (dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(D=127), dict(D=2048), dict(rot=0), dict(rot=63),
               dict(rot=130), dict(layout=2), dict(backward=2), dict(m=float("nan")), dict(q=None),
               dict(k=None), dict(pos=None), dict(freq=None), dict(qo=None), dict(ko=None),
               dict(q=FAKE + 2), dict(pos=FAKE + 2)):
        assert call(**kw) == binding.GDN_ERR_INVALID_ARG, kw
    assert call(T=0, q=None, k=None) == binding.GDN_OK


@pytest.mark.parametrize("rot", [2, 24, 128])
def test_rope_frequencies(rot):
    i = np.arange(rot // 2)
    f = 10000.0 ** (-2.0 * i / rot) / (2 * np.pi)
    kept = np.clip((f * 4096 - 1.0) / 31.0, 0, 1)
    for kind, want in (("none", f), ("linear", f / 8), ("parts", f * kept + f / 8 * (1 - kept))):
        got = gdn.rope_frequencies(rot, scaling=kind, factor=8.0, trained_len=4096, device="cpu").double()
        assert got.shape == (2, rot // 2)
        # head + tail hold 48 bits; pow and the division are good to a few 2^-53
        np.testing.assert_allclose(got.sum(0).numpy(), want, rtol=2.0 ** -46, atol=0)
    for kw in (dict(base=1.0), dict(scaling="linear", factor=0.5), dict(scaling="parts", factor=2.0),
               dict(scaling="parts", factor=2.0, trained_len=4096, low_turns=4.0, high_turns=4.0)):
        with pytest.raises(gdn.GdnError):
            gdn.rope_frequencies(rot, device="cpu", **kw)
    assert gdn.gdn_rope_frequencies(3, 1e4, 0, 1.0, 0.0, 1.0, 32.0, (ctypes.c_float * 4)()) \
        == binding.GDN_ERR_INVALID_ARG
    assert gdn.gdn_rope_frequencies(4, 1e4, 3, 1.0, 0.0, 1.0, 32.0, (ctypes.c_float * 4)()) \
        == binding.GDN_ERR_INVALID_ARG


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
    cu = np.array([0, 6], np.int32)
    seq = dict(q=(bf, (6, 2, 128)), k=(bf, (6, 2, 128)), v=(bf, (6, 4, 128)), log_decay=(f32, (4,)),
               cu_dev=(i32, (2,)), device_status=(i32, (1,)))
    state = (f32, (1, 4, 128, 128))
    pool = dict(state_pool=(f32, (3, 4, 128, 128)), state_indices=(i32, (1,)))
    step = {n: seq[n] for n in ("q", "k", "v", "log_decay", "device_status")}
    yield gdn.linear_attn_fwd, dict(seq, initial_state=state, workspace=(torch.uint8, (64,))), dict(cu_host=cu)
    yield gdn.linear_attn_bwd, dict(seq, d_o=(bf, (6, 4, 128)), initial_state=state, d_final_state=state,
                                    workspace=(torch.uint8, (64,))), dict(cu_host=cu)
    yield gdn.linear_attn_prefill_paged, dict(seq, **pool, has_initial_state=(i32, (1,)), problem_status=(i32, (1,)),
                                              workspace=(torch.uint8, (64,))), dict(cu_host=cu)
    yield gdn.linear_attn_step, dict(step, state_pool=(f32, (3, 4, 128, 128)), state_indices=(i32, (6,))), {}
    yield gdn.rope, dict(q=(bf, (6, 2, 128)), k=(bf, (6, 2, 128)), positions=(i32, (6,)), freq=(f32, (2, 32))), {}


def test_tensors_of_another_device_are_refused(monkeypatch):
    class Refused(Exception):
        pass

    class Library:
        def __getattr__(self, name):
            def launch(*args):
                raise Refused(name)
            return launch

    linear._ready()
    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(linear, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(linear, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch, "empty_like", lambda t: t)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: _Elsewhere(torch.float32, a[0]))
    for call, tensors, rest in _calls():
        with pytest.raises(Refused):   # all on the current device: the call goes through
            call(**{n: _Elsewhere(*x) for n, x in tensors.items()}, **rest)
        for other in tensors:
            for device in (1, -1):
                with pytest.raises((ValueError, TypeError), match="device|CUDA"):
                    call(**{n: _Elsewhere(*x, device=device if n == other else 0) for n, x in tensors.items()},
                         **rest)
        with pytest.raises(ValueError, match="device"):   # all of them on one that is not current
            call(**{n: _Elsewhere(*x, device=1) for n, x in tensors.items()}, **rest)


def _torch_rope(q, k, positions, freq, layout="half", mscale=1.0, backward=False, inplace=False):
    """gdn.rope in torch operations (half layout), as opaque to autograd as the kernel."""
    def turn(x):
        a = 2 * np.pi * positions.double()[:, None] * freq.double().sum(0)
        c, s = (mscale * f(a)[:, None].to(x.dtype) for f in (torch.cos, torch.sin))
        half = freq.shape[1]
        one, two, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
        s = -s if backward else s
        return torch.cat([one * c - two * s, two * c + one * s, rest], -1)
    with torch.no_grad():
        return turn(q), None if k is None else turn(k)


def test_rotary_has_a_second_derivative(monkeypatch):
    # a penalty on a gradient that passed the rotation keeps its own gradient
    monkeypatch.setattr(linear, "rope", _torch_rope)
    rng = torch.Generator().manual_seed(1)
    q, k = (torch.randn(5, h, 8, generator=rng, dtype=torch.float64, requires_grad=True) for h in (2, 1))
    pos, freq = torch.arange(5, dtype=torch.int32), torch.rand(2, 3, generator=rng)
    assert torch.autograd.gradcheck(lambda x, y: gdn.rotary(x, y, pos, freq, mscale=1.25), (q, k))
    assert torch.autograd.gradgradcheck(lambda x, y: gdn.rotary(x, y, pos, freq, mscale=1.25), (q, k))


@pytest.mark.parametrize("which", ["linear_attention", "chunk_gated_delta_rule"])
def test_second_derivatives_that_do_not_exist_are_refused(monkeypatch, which):
    # the gradients of a fused backward are not differentiable: a loss on them must not lose its term
    x = torch.randn(4, 1, 128, requires_grad=True)
    zeros = {n: torch.zeros(4, 1, 128) for n in ("dq", "dk", "dv")}
    if which == "linear_attention":
        monkeypatch.setattr(linear, "linear_attn_fwd", lambda *a, **kw: (a[2] * 2.0, None))
        monkeypatch.setattr(linear, "linear_attn_bwd", lambda *a, **kw: dict(zeros, dh0=None))
        o, _ = gdn.linear_attention(x, x, x, torch.zeros(1), cu_seqlens=torch.tensor([0, 4]))
    else:
        monkeypatch.setattr(binding, "chunk_fwd", lambda *a, **kw: (a[2] * 2.0, None, None))
        monkeypatch.setattr(binding, "chunk_bwd", lambda *a, **kw: dict(zeros, dg=torch.zeros(4, 1),
                                                                        dbeta=torch.zeros(4, 1), dh0=None))
        g = torch.zeros(4, 1, requires_grad=True)
        o, _ = gdn.chunk_gated_delta_rule(x, x, x, g, g, cu_seqlens=torch.tensor([0, 4]))
    (dx,) = torch.autograd.grad(o.float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once more"):
        (dx.square().sum() + o.sum()).backward()


def test_rotary_refuses_a_gradient_of_the_frequencies(monkeypatch):
    monkeypatch.setattr(linear, "rope", _torch_rope)
    q = torch.randn(5, 2, 8, requires_grad=True)
    with pytest.raises(ValueError, match="freq"):
        gdn.rotary(q, q, torch.arange(5, dtype=torch.int32), torch.rand(2, 3, requires_grad=True))
    with torch.no_grad():
        gdn.rotary(q, q, torch.arange(5, dtype=torch.int32), torch.rand(2, 3, requires_grad=True))


def test_rotary_without_k(monkeypatch):
    monkeypatch.setattr(linear, "rope", _torch_rope)
    q = torch.randn(5, 2, 8, requires_grad=True)
    pos, freq = torch.arange(5, dtype=torch.int32), torch.rand(2, 3)
    y, none = gdn.rotary(q, None, pos, freq)
    both, _ = gdn.rotary(q, q, pos, freq)
    assert none is None and torch.equal(y, both)
    (dq,) = torch.autograd.grad(y, q, torch.ones_like(y))
    assert torch.equal(dq, _torch_rope(torch.ones_like(y), None, pos, freq, backward=True)[0])


def test_rope_in_place_shows_itself_to_autograd(monkeypatch):
    class Library:
        def gdn_rope(self, *args):
            return binding.GDN_OK

    linear._ready()
    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(linear, "_device", lambda q: -1)   # host tensors stand in; nothing is launched
    monkeypatch.setattr(linear, "_raw_stream", lambda device: 0)
    q, k = (torch.zeros(3, h, 8, dtype=torch.bfloat16) for h in (2, 1))
    pos, freq = torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4)
    before = q._version, k._version
    gdn.rope(q, k, pos, freq)
    assert (q._version, k._version) == before
    gdn.rope(q, k, pos, freq, inplace=True)
    assert q._version > before[0] and k._version > before[1]
    # a tensor that a graph has saved cannot change unseen
    w = torch.ones(8, dtype=torch.bfloat16, requires_grad=True)
    loss = (q * w).sum()
    gdn.rope(q, None, pos, freq, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # nor one whose gradient is asked for, unless none is recorded
    x = q.clone().requires_grad_()
    for args in ((x, None), (q, k.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            gdn.rope(*args, pos, freq, inplace=True)
        with torch.no_grad():
            gdn.rope(*args, pos, freq, inplace=True)
    with torch.inference_mode():
        gdn.rope(torch.zeros(3, 2, 8, dtype=torch.bfloat16), None, pos, freq, inplace=True)


def test_offsets_changed_before_the_backward(monkeypatch):
    # a loop that reuses its offset buffers: the backward has the forward's host copy, and a device
    # copy that changed in place is an error
    seen = []
    monkeypatch.setattr(linear, "linear_attn_fwd", lambda *a, **kw: (a[2] * 2.0, None))
    monkeypatch.setattr(linear, "linear_attn_bwd", lambda q, k, v, g, do, cu, cu_dev, **kw: (
        seen.append(cu.copy()), dict(dq=q * 0, dk=k * 0, dv=v * 0, dh0=None))[1])
    x = torch.randn(4, 1, 128, requires_grad=True)
    host, dev = torch.tensor([0, 1, 4], dtype=torch.int32), torch.tensor([0, 1, 4], dtype=torch.int32)
    o, _ = gdn.linear_attention(x, x, x, torch.zeros(1), cu_seqlens=dev, cu_seqlens_cpu=host)
    host[1] = 3
    o.float().sum().backward()
    assert seen[0].tolist() == [0, 1, 4]
    o, _ = gdn.linear_attention(x, x, x, torch.zeros(1), cu_seqlens=dev, cu_seqlens_cpu=host)
    dev[1] = 3
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.float().sum().backward()


def test_packed_problem_is_the_structure(monkeypatch):
    linear._ready()
    cu = np.array([0, 2, 6], np.int32)
    tensors = [_Elsewhere(torch.int32, (3,)), _Elsewhere(torch.int32, (1,))]
    tensors[1].data_ptr = lambda: FAKE + 4
    raw, keep, N = linear._problem((6, 2, 128, 4, 128), cu, tensors[0], 0.5, tensors[1], 7, 0)
    p = binding.GdnProblem.from_buffer_copy(raw)
    assert len(raw) == ctypes.sizeof(binding.GdnProblem) and N == 2 and keep is cu
    got = {n: getattr(p, n) for n, _ in binding.GdnProblem._fields_ if n != "cu_seqlens_host"}
    assert got == dict(num_seqs=2, total_tokens=6, num_k_heads=2, num_v_heads=4, head_dim_k=128, head_dim_v=128,
                       scale=0.5, beta_dtype=0, cu_seqlens_dev=FAKE, device_status=FAKE + 4, scan_segment_chunks=7)
    assert ctypes.addressof(p.cu_seqlens_host.contents) == cu.ctypes.data
    # a further field would change the format, and the packing would raise
    class Longer(ctypes.Structure):
        _fields_ = binding.GdnProblem._fields_ + [("more", ctypes.c_int32)]
    assert linear._struct_of(Longer).format != linear._PROBLEM.format
