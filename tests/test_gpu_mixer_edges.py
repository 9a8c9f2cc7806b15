"""The convolution, the scan and the norms where calls meet: values that are no numbers, gradients that are parts
of tensors, training steps in graphs, calls on two streams, one workspace for two graphs, offsets past 32 bits."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, t=BF: torch.randn(*s, generator=g, device="cuda", dtype=F32).to(t)


def _cu(lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


def _scan(lens, C, Ns=16, G=1, seed=0, t=BF):
    rn, T = _gen(seed), sum(lens)
    return dict(x=rn(T, C, t=t), dt=rn(T, C, t=t), A_log=rn(C, Ns, t=F32) / 2, B=rn(T, G, Ns, t=t), C=rn(T, G, Ns, t=t), D=rn(C, t=F32),
                z=rn(T, C, t=t), dt_bias=rn(C, t=F32) - 2), rn(T, C, t=t)


@pytest.mark.parametrize("seg", [-1, 32])
def test_a_rate_that_is_no_number_shows(seg):
    a, dy = _scan([70, 30], 40)
    a["A_log"][7, 3] = float("nan")
    cu, cu_dev = _cu([70, 30])
    y, ht = gdn.selective_scan_fwd(**a, cu_host=cu, cu_dev=cu_dev, segment_tokens=seg)
    others = [c for c in range(40) if c != 7]
    # (the first token has no state to decay but zeros: 0 NaN)
    assert torch.isnan(y[:, 7]).all() and torch.isfinite(y[:, others]).all()
    assert torch.isnan(ht[:, 7, 3]).all() and torch.isfinite(ht[:, others]).all() and torch.isfinite(ht[:, 7, :3]).all()
    got = gdn.selective_scan_bwd(**a, dy=dy, cu_host=cu, cu_dev=cu_dev, segment_tokens=seg)
    assert torch.isnan(got["dA_log"][7, 3]) and torch.isnan(got["ddt"][:, 7]).all()
    assert torch.isfinite(got["dx"][:, others]).all() and torch.isfinite(got["dA_log"][others]).all()
    pool = torch.zeros(3, 40, 16, device="cuda")
    idx = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    one = {k: v[:2] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    y = gdn.selective_scan_step(**one, state_pool=pool, state_indices=idx)
    assert torch.isnan(y[:, 7]).all() and torch.isfinite(y[:, others]).all()


@pytest.mark.parametrize("seg", [-1, 64])
def test_tokens_without_a_step_leave_the_state(seg):
    a, dy = _scan([1000, 13], 40)
    a["dt"].fill_(-300.0)   # softplus is 0
    cu, cu_dev = _cu([1000, 13])
    h0 = _gen(9)(2, 40, 16, t=F32)
    y, ht = gdn.selective_scan_fwd(**a, cu_host=cu, cu_dev=cu_dev, initial_state=h0, segment_tokens=seg)
    assert torch.equal(ht, h0)
    got = gdn.selective_scan_bwd(**a, dy=dy, cu_host=cu, cu_dev=cu_dev, initial_state=h0, d_final_state=h0, segment_tokens=seg)
    assert not got["dB"].any() and not got["ddt"].any() and not got["dA_log"].any()
    pool = torch.cat([torch.zeros_like(h0[:1]), h0])
    idx = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    one = {k: v[:2] if k in ("x", "dt", "B", "C", "z") else v for k, v in a.items()}
    for _ in range(3):
        gdn.selective_scan_step(**one, state_pool=pool, state_indices=idx)
    assert torch.equal(pool[1:], h0)


def test_a_long_memory_does_not_drift():
    # steps of 0.001 .. 0.01 and rates near 1: after 2000 tokens a state keeps a part of its start, and what its
    # decays are off by on average shows 2000 times
    a, _ = _scan([2000], 64, 8, t=F32)
    a["A_log"] *= 0.2
    a["dt"].zero_()
    a["x"].zero_()
    step = torch.linspace(0.001, 0.01, 64, device="cuda", dtype=torch.float64)
    a["dt_bias"] = torch.log(torch.expm1(step)).float()
    h0 = 1 + _gen(2)(1, 64, 8, t=F32).abs()
    cu, cu_dev = _cu([2000])
    _, ht = gdn.selective_scan_fwd(**a, cu_host=cu, cu_dev=cu_dev, initial_state=h0, segment_tokens=-1)
    d = torch.nn.functional.softplus(a["dt_bias"].double(), threshold=40)
    total = 2000 * d[:, None] * torch.exp(a["A_log"].double())
    want = h0.double() * torch.exp(-total)
    off = ht[0].double() / want[0] - 1
    # Every token of a state has the same decay here, so that its errors are no random ones: the exponential's
    # 2^-22 and what it is lifted by, below 2^-25, and the state's own rounding, 2^-24, are below 2^-21.4 a token, all
    # 2000 times; d is off by 2^-19 (as in the definition's bounds), A and its products by 2^-22, of the whole decay.
    assert (off.abs() <= 2000 * 2.0 ** -21.4 + total * (2.0 ** -19 + 2.0 ** -22)).all()
    # Of 512 states with errors of 3e-8 a token the mean is off by 3e-8 / 512^0.5 = 1.3e-9: what is left is the bias,
    # which is 1.6e-8 for these steps without the lift and within 2e-9 of nothing with it.
    assert abs(float(off.mean())) <= 2000 * (2e-9 + 4 * 1.3e-9)


@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_a_gate_that_is_no_number_shows(gate):
    rn = _gen()
    x, z, dy, w = rn(4, 64), rn(4, 64), rn(4, 64), rn(64, t=F32)
    z[2, 5] = float("nan")
    y, _ = gdn.rms_norm_fwd(x, w, z=z, gate=gate)
    got = gdn.rms_norm_bwd(x, w, dy, z=z, gate=gate)
    assert torch.isnan(y[2, 5]) and torch.isnan(got["dz"][2, 5]) and torch.isnan(got["dweight"][5])
    assert torch.isnan(got["dx"][2]).all()   # (through the row's mean)
    rest = [0, 1, 3]
    for t in (y, got["dz"], got["dx"]):
        assert torch.isfinite(t[rest]).all()


@pytest.mark.parametrize("t", [BF, F32])
def test_gradients_that_are_parts_of_tensors(t):
    # a row's five elements are no 16 bytes: what the joined tensor's gradient gives starts anywhere
    rn, lens = _gen(), [3, 4]
    cu, cu_dev = _cu(lens)
    kw = dict(cu_seqlens=cu_dev, cu_seqlens_cpu=cu)
    x, h0, up = rn(7, 5, t=t), rn(3, 5, 3, t=t)[1:], rn(10, 5, t=t)
    w = rn(5, 4, t=F32)

    def check(f, g, tensors):
        leaves = [v.detach().clone().requires_grad_() for v in tensors]
        whole = [v.detach().clone().requires_grad_() for v in tensors]
        out = torch.cat([up[:3], f(*leaves)])
        out.backward(up)
        g(*whole).backward(up[3:].clone())
        for a, b in zip(leaves, whole):
            assert torch.equal(a.grad, b.grad)
    conv = lambda x: gdn.short_conv(x, w, initial_state=h0, **kw)[0]  # noqa: E731
    check(conv, conv, [x])
    a, _ = _scan(lens, 5, 8, t=t)
    s0 = rn(3, 5, 8, t=F32)[1:]
    scan = lambda x, B: gdn.selective_scan(x, a["dt"], a["A_log"], B, a["C"], z=a["z"], initial_state=s0, **kw)[0]  # noqa: E731
    check(scan, scan, [a["x"], a["B"]])
    vec = rn(6, t=F32)[1:]
    check(lambda x, z: gdn.rms_norm(x, vec, z=z), lambda x, z: gdn.rms_norm(x, vec.clone(), z=z), [x, rn(7, 5, t=t)])
    # and inputs that are parts
    wide = rn(8, 5, t=t)
    assert wide[1:].data_ptr() % 16
    assert torch.equal(gdn.rms_norm(wide[1:], vec), gdn.rms_norm(wide[1:].clone(), vec))
    assert torch.equal(gdn.rms_norm(wide[1:], vec, residual=wide[1:])[1], wide[1:] + wide[1:])


def test_a_training_step_in_a_graph():
    lens, C = [33, 0, 90], 64
    cu, cu_dev = _cu(lens)
    kw = dict(cu_seqlens=cu_dev, cu_seqlens_cpu=cu)
    a, dy = _scan(lens, C)
    rn = _gen(3)
    params = [rn(C, 4, t=F32), rn(C, t=F32), a["A_log"], a["D"], a["dt_bias"], rn(C, t=F32)]
    params = [p.clone().requires_grad_() for p in params]
    x = a["x"].clone().requires_grad_()

    def step():
        w, b, A_log, D, bias, norm = params
        u = gdn.short_conv(x, w, b, **kw)[0]
        y = gdn.selective_scan(u, a["dt"], A_log, a["B"], a["C"], D=D, z=a["z"], dt_bias=bias, **kw)[0]
        y, _ = gdn.rms_norm(y, norm, z=a["z"], residual=x)
        return torch.autograd.grad(y, [x, *params], dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (5, 6):
        with torch.no_grad():
            x.copy_(_gen(seed)(*x.shape))
            for p in params:
                p.add_(0.1)
        graph.replay()
        held = [g.clone() for g in got]
        for g, want in zip(held, step()):
            assert torch.equal(g, want)


def test_two_streams_at_once_and_a_workspace_of_two_graphs():
    lens, C = [900, 60], 96
    cu, cu_dev = _cu(lens)
    calls = [_scan(lens, C, seed=s) for s in (1, 2)]
    run = lambda a, dy, **kw: (gdn.selective_scan_fwd(**a, cu_host=cu, cu_dev=cu_dev, segment_tokens=64, **kw)[0],  # noqa: E731
                               *gdn.selective_scan_bwd(**a, dy=dy, cu_host=cu, cu_dev=cu_dev, segment_tokens=64, **kw).values())
    want = [[t.clone() for t in run(a, dy)] for a, dy in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, (a, dy) in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(run(a, dy))
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(i, j) for i, j in zip(w, g))
    # graphs that are replayed one after another may have one workspace
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    graphs = []
    for a, dy in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(a, dy, workspace=ws)
        graphs.append((graph, out))
    for _ in range(3):
        for w, (graph, out) in zip(want, graphs):
            graph.replay()
            assert all(torch.equal(i, j) for i, j in zip(w, out))


def test_a_workspace_that_is_too_small_is_refused():
    a, dy = _scan([300], 32)
    cu, cu_dev = _cu([300])
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for f in (lambda: gdn.selective_scan_fwd(**a, cu_host=cu, cu_dev=cu_dev, segment_tokens=64, workspace=small),
              lambda: gdn.selective_scan_bwd(**a, dy=dy, cu_host=cu, cu_dev=cu_dev, workspace=small),
              lambda: gdn.short_conv_bwd(a["x"], torch.ones(32, 4, device="cuda"), dy, cu, cu_dev, workspace=small),
              lambda: gdn.rms_norm_bwd(a["x"], torch.ones(32, device="cuda"), dy, workspace=small[:64])):
        with pytest.raises(gdn.GdnError) as e:
            f()
        assert e.value.status == gdn.binding.GDN_ERR_WORKSPACE_TOO_SMALL


# ------------------------------------------------------------------------------ offsets past 32 bits
LAST = 10   # tokens of the last sequence, or rows, whose results are those of a call of their own


def _much(*shape):
    return torch.randn(*shape, device="cuda", dtype=BF)


def test_convolution_past_32_bits():
    C, lens = 32768, [70000, LAST]
    cu, cu_dev = _cu(lens)
    x, w = _much(sum(lens), C), torch.randn(C, 4, device="cuda")
    assert x.numel() > 1 << 31
    few = (x[-LAST:].clone(), w), _cu([LAST])
    y, ht = gdn.short_conv_fwd(x, w, cu, cu_dev)
    want, last = gdn.short_conv_fwd(*few[0], *few[1])
    assert torch.equal(y[-LAST:], want) and torch.equal(ht[1:], last)
    got = gdn.short_conv_bwd(x, w, y, cu, cu_dev)
    want = gdn.short_conv_bwd(*few[0], want, *few[1])
    assert torch.equal(got["dx"][-LAST:], want["dx"]) and torch.equal(got["dh0"][1:], want["dh0"])
    del x, y, got
    # a slot far into a pool
    slots = (1 << 31) // (C * 3) + 5
    pool = torch.zeros(slots, C, 3, device="cuda", dtype=BF)
    pool[-1] = last[0]
    near = torch.cat([torch.zeros_like(last), last])
    at = lambda i: torch.tensor([i], dtype=torch.int32, device="cuda")  # noqa: E731
    x = few[0][0]
    y = gdn.short_conv_prefill_paged(x, w, *few[1], pool, at(slots - 1))
    want = gdn.short_conv_prefill_paged(x, w, *few[1], near, at(1))
    assert torch.equal(y, want) and torch.equal(pool[-1], near[1])
    y = gdn.short_conv_step(x[:1], w, pool, at(slots - 1))
    want = gdn.short_conv_step(x[:1], w, near, at(1))
    assert torch.equal(y, want) and torch.equal(pool[-1], near[1]) and not pool[:-1].any()


def test_scan_past_32_bits():
    C, lens = 32768, [70000, LAST]
    cu, cu_dev = _cu(lens)
    T, Ns = sum(lens), 16
    x, dt, B, Cm = _much(T, C), _much(T, C), _much(T, 1, Ns), _much(T, 1, Ns)
    A_log, bias = torch.randn(C, Ns, device="cuda") / 2, torch.randn(C, device="cuda") - 2
    few = [t[-LAST:].clone() for t in (x, dt, B, Cm)]
    fwd = lambda x, dt, B, Cm, *cu, **kw: gdn.selective_scan_fwd(x, dt, A_log, B, Cm, *cu, dt_bias=bias, **kw)  # noqa: E731
    bwd = lambda x, dt, B, Cm, dy, *cu, **kw: gdn.selective_scan_bwd(x, dt, A_log, B, Cm, dy, *cu, dt_bias=bias, **kw)  # noqa: E731
    y, ht = fwd(x, dt, B, Cm, cu, cu_dev, segment_tokens=512)
    want, last = fwd(*few, *_cu([LAST]))
    assert torch.equal(y[-LAST:], want) and torch.equal(ht[1:], last)
    got = bwd(x, dt, B, Cm, y, cu, cu_dev, segment_tokens=512)
    want = bwd(*few, want, *_cu([LAST]))
    for n in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(got[n][-LAST:], want[n]), n
    assert torch.equal(got["dh0"][1:], want["dh0"])
    del x, dt, y, got
    slots = (1 << 31) // (C * Ns) + 5
    pool = torch.zeros(slots, C, Ns, device="cuda")
    pool[-1] = last[0]
    near = torch.cat([torch.zeros_like(last), last])
    at = lambda i: torch.tensor([i], dtype=torch.int32, device="cuda")  # noqa: E731
    paged = lambda p, i: gdn.selective_scan_prefill_paged(few[0], few[1], A_log, *few[2:], *_cu([LAST]), p, at(i), dt_bias=bias)  # noqa: E731
    step = lambda p, i: gdn.selective_scan_step(few[0][:1], few[1][:1], A_log, few[2][:1], few[3][:1], p, at(i), dt_bias=bias)  # noqa: E731
    for f in (paged, step):
        assert torch.equal(f(pool, slots - 1), f(near, 1)) and torch.equal(pool[-1], near[1])
    assert not pool[:-1].any()


def test_norm_past_32_bits():
    D, rows = 4096, (1 << 31) // 4096 + LAST
    x, z, w = _much(rows, D), _much(rows, D), torch.randn(D, device="cuda")
    y, h = gdn.rms_norm_fwd(x, w, z=z, residual=x)
    want, few = gdn.rms_norm_fwd(x[-LAST:].clone(), w, z=z[-LAST:].clone(), residual=x[-LAST:].clone())
    assert torch.equal(y[-LAST:], want) and torch.equal(h[-LAST:], few)
    got = gdn.rms_norm_bwd(h, w, y, z=z, dh=x)
    want = gdn.rms_norm_bwd(few, w, want, z=z[-LAST:].clone(), dh=x[-LAST:].clone())
    for n in ("dx", "dz"):
        assert torch.equal(got[n][-LAST:], want[n]), n
