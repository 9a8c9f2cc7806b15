"""The selective scan on the GPU against its 64-bit definition: state sizes, groups, types, packs with
empty and short sequences, split plans, pools, steps, gradients, strided rows, extreme inputs."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import mixer_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, lens, C, Ns=16, G=1, dtype=BF, gate=True, skip=True, bias=True, seed=0, wider=0, rate=0.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rn = lambda *s, t=dtype, k=1.0: (torch.randn(*s, generator=g, device="cuda") * k).to(t)  # noqa: E731
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.cu_dev = torch.from_numpy(self.cu).cuda()
        T, N = int(self.cu[-1]), len(lens)
        cut = lambda n: rn(T, n + wider)[:, wider // 2:wider // 2 + n]  # noqa: E731
        self.x, self.dt, self.z = cut(C), cut(C), cut(C) if gate else None
        self.B, self.C = (cut(G * Ns).unflatten(1, (G, Ns)) for _ in range(2))
        self.A_log = torch.log(torch.arange(1, Ns + 1, device="cuda").float()) + rn(C, Ns, t=F32, k=0.2) + rate
        self.D = rn(C, t=F32) if skip else None
        # steps from about 0.002 to 2
        self.bias = rn(C, t=F32, k=2.0) - 3.0 if bias else None
        self.h0, self.dht, self.dy = rn(N, C, Ns, t=F32), rn(N, C, Ns, t=F32), rn(T, C)
        self.t = dtype

    def args(self):
        return self.x, self.dt, self.A_log, self.B, self.C

    def kw(self, **more):
        return dict(D=self.D, z=self.z, dt_bias=self.bias, **more)

    def fwd(self, **kw):
        return gdn.selective_scan_fwd(*self.args(), self.cu, self.cu_dev, **self.kw(initial_state=self.h0, **kw))

    def bwd(self, **kw):
        return gdn.selective_scan_bwd(*self.args(), self.dy, self.cu, self.cu_dev,
                                      **self.kw(initial_state=self.h0, d_final_state=self.dht, **kw))

    def reference(self, grads=False):
        return ref.scan(*self.args(), self.cu, self.D, self.z, self.bias, self.h0, self.dy if grads else None,
                        self.dht if grads else None)

    def check(self, got, want, names):
        for name in names:
            value, off = want[name]
            t = F32 if name in ("ht", "dA_log", "dD", "ddt_bias", "dh0") else self.t
            ref.check(name, got[name], value, off + ref.HALF[t] * value.abs() + 1e-30)


GRADS = ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
SHAPES = [([5], 8, 16, 1), ([1], 1, 8, 1), ([0, 1, 2, 9, 0, 33, 70], 64, 16, 2), ([64, 65, 1], 96, 32, 3), ([3, 0], 7, 8, 7),
          ([100, 17], 130, 16, 1), ([1] * 20, 16, 32, 1), ([40], 1100, 8, 2), ([31], 264, 16, 3)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens, C, Ns, G", SHAPES)
def test_forward_and_gradient(lens, C, Ns, G, dtype):
    for there in (True, False):
        c = Case(lens, C, Ns, G, dtype, there, there, there, seed=C)
        want = c.reference(grads=True)
        y, ht = c.fwd()
        c.check(dict(y=y, ht=ht), want, ("y", "ht"))
        got = c.bwd()
        assert [n for n in GRADS if got[n] is None] == ([] if there else ["dD", "dz", "ddt_bias"])
        c.check(got, want, [n for n in GRADS if got[n] is not None])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens, C, Ns, seg", [([97], 64, 16, 32), ([200, 0, 31, 65], 40, 8, 32), ([64, 33], 32, 32, 64),
                                              ([130, 1, 70], 16, 16, 96), ([257], 70, 16, 33)])
def test_split_scans(lens, C, Ns, seg, dtype):
    # slow decays too, so that the states pass through the segments
    for rate in (0.0, -4.0):
        c = Case(lens, C, Ns, 2, dtype, seed=seg, rate=rate)
        want = c.reference(grads=True)
        y, ht = c.fwd(segment_tokens=seg)
        c.check(dict(y=y, ht=ht), want, ("y", "ht"))
        c.check(c.bwd(segment_tokens=seg), want, GRADS)
        # over slots, the same bits
        N = len(lens)
        pool = torch.randn(N + 2, C, Ns, device="cuda")
        idx = torch.arange(N, 0, -1, dtype=torch.int32, device="cuda")
        pool[idx.long()] = c.h0
        before = pool.clone()
        yp = gdn.selective_scan_prefill_paged(*c.args(), c.cu, c.cu_dev, pool, idx, segment_tokens=seg, **c.kw())
        assert torch.equal(yp, y) and torch.equal(pool[idx.long()], ht)
        assert torch.equal(pool[[0, N + 1]], before[[0, N + 1]])


def test_gradient_against_differences():
    c = Case([20, 13], 12, 8, 2, F32, seed=3)
    got = c.bwd()
    names = dict(x="dx", dt="ddt", A_log="dA_log", B="dB", C="dC", D="dD", z="dz", bias="ddt_bias", h0="dh0")

    def loss():
        want = c.reference()
        return float((want["y"][0] * c.dy.double()).sum() + (want["ht"][0] * c.dht.double()).sum())
    for field, name in names.items():
        at = getattr(c, field)
        step, eps = torch.randn_like(at).double(), 1e-5
        ends = []
        for sign in (1, -1):
            setattr(c, field, at.double() + sign * eps * step)
            ends.append(loss())
        setattr(c, field, at)
        want, mine = (ends[0] - ends[1]) / (2 * eps), float((got[name].double() * step).sum())
        # central differences: eps^2 of the third derivative; the gradient: fp32 sums, 2^-14 of their magnitude
        size = float((got[name].double() * step).abs().sum())
        assert abs(mine - want) <= 2.0 ** -14 * size + 1e-6 * (1 + abs(want)), name


def test_the_library_s_own_plan():
    # one long sequence of few channels is split, and agrees with the unsplit walk
    c = Case([5000], 32, 16, 1, F32, rate=-5.0)
    y, ht = c.fwd()
    y1, ht1 = c.fwd(segment_tokens=-1)
    # both are within (n + 4) 2^-21 + 2^-17 of sums whose terms are of the order of their values
    for a, b in ((y, y1), (ht, ht1)):
        assert float((a - b).norm() / b.norm()) < 2 * 5004 * 2.0 ** -21
    got, want = c.bwd(), c.bwd(segment_tokens=-1)
    for n in GRADS:
        assert float((got[n] - want[n]).norm() / want[n].norm()) < 4 * 5004 * 2.0 ** -21, n


@pytest.mark.parametrize("C, wider", [(64, 16), (64, 3), (33, 31)])
def test_rows_that_lie_apart(C, wider):
    c, d = Case([70, 9], C, wider=wider), Case([70, 9], C, wider=wider)
    for n in ("x", "dt", "z", "B", "C"):
        setattr(d, n, getattr(d, n).contiguous())
    for a, b in zip((*c.fwd(), *c.bwd().values()), (*d.fwd(), *d.bwd().values())):
        assert torch.equal(a, b)
    pool = torch.randn(80, C, 16, device="cuda")
    idx = torch.arange(79, dtype=torch.int32, device="cuda") + 1
    p, q = pool.clone(), pool.clone()
    assert torch.equal(gdn.selective_scan_step(*c.args(), p, idx, **c.kw()),
                       gdn.selective_scan_step(*d.args(), q, idx, **d.kw())) and torch.equal(p, q)


def test_slots_that_are_none_or_outside_or_fresh():
    c = Case([4, 5, 6, 0], 16)
    pool = torch.randn(5, 16, 16, device="cuda")
    before, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([0, 5, 2, 4], dtype=torch.int32, device="cuda")
    resume = torch.tensor([1, 1, 0, 1], dtype=torch.int32, device="cuda")
    y = gdn.selective_scan_prefill_paged(*c.args(), c.cu, c.cu_dev, pool, idx, resume, device_status=status, **c.kw())
    c.h0[:3], c.h0[3] = 0, before[4]
    want, last = c.fwd()
    assert torch.equal(y, want) and int(status) == 1
    assert torch.equal(pool[2], last[2]) and torch.equal(pool[[0, 1, 3, 4]], before[[0, 1, 3, 4]])
    status.zero_()
    c = Case([4], 40, 8, 2)
    pool = torch.randn(3, 40, 8, device="cuda")
    before = pool.clone()
    idx = torch.tensor([-1, 1, 3, 0], dtype=torch.int32, device="cuda")
    y = gdn.selective_scan_step(*c.args(), pool, idx, device_status=status, **c.kw())
    assert int(status) == 1 and not y[[0, 2, 3]].any() and y[1].any()
    assert torch.equal(pool[[0, 2]], before[[0, 2]]) and not torch.equal(pool[1], before[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C, Ns, G", [(8, 16, 1), (1, 8, 1), (260, 32, 2), (1031, 16, 1)])
def test_steps_are_the_forward(C, Ns, G, dtype):
    c = Case([5, 5, 5], C, Ns, G, dtype)
    want = c.reference()
    pool = torch.zeros(5, C, Ns, device="cuda")
    idx = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    pool[idx.long()] = c.h0
    at = lambda t, i: t.reshape(3, 5, *t.shape[1:])[:, i].contiguous()  # noqa: E731
    y = []
    for i in range(5):
        x, dt, B, Cm, z = (at(t, i) for t in (c.x, c.dt, c.B, c.C, c.z))
        y.append(gdn.selective_scan_step(x, dt, c.A_log, B, Cm, pool, idx, D=c.D, z=z, dt_bias=c.bias))
    c.check(dict(y=torch.stack(y, 1).reshape(15, C), ht=pool[idx.long()]), want, ("y", "ht"))


def test_no_tokens_and_no_rows():
    c = Case([0, 0], 16)
    y, ht = c.fwd()
    assert y.shape == (0, 16) and torch.equal(ht, c.h0)
    got = c.bwd()
    assert torch.equal(got["dh0"], c.dht) and not got["dA_log"].any() and not got["dD"].any()
    pool = torch.randn(2, 16, 16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert gdn.selective_scan_step(*c.args(), pool, none, **c.kw()).shape == (0, 16)


def test_extreme_steps_and_rates():
    c = Case([30], 8, 8, 1, F32, bias=False)
    c.dt[:, 0], c.dt[:, 1], c.dt[:, 2], c.dt[:, 3] = -80.0, 60.0, -15.0, 19.9
    c.A_log[4], c.A_log[5], c.A_log[6] = 200.0, -200.0, float("-inf")   # each token alone; no decay at all
    want = Case.reference(c)
    y, ht = c.fwd()
    for v in (y, ht):
        assert torch.isfinite(v).all()
    # (e^200 in the reference is finite in 64 bits, its decays are 0 as here)
    c.check(dict(y=y, ht=ht), want, ("y", "ht"))
    # rates beyond fp32 have no gradient to compare
    got = c.bwd()
    assert all(torch.isfinite(got[n]).all() for n in ("dx", "dB", "dC", "dh0"))


def test_infinities_stay_in_their_channel():
    c = Case([40, 30], 16, 16, 1, gate=False)
    c.x[10, 3] = float("inf")
    c.x[69, 5] = float("nan")
    y, ht = c.fwd()
    bad = ~torch.isfinite(y)
    assert bad[10, 3] and bad[69, 5] and not bad[40:69].any()
    bad[:, 3], bad[:, 5] = False, False
    assert not bad.any() and not (~torch.isfinite(ht))[:, [0, 1, 2, 4, 6, 7]].any()


def test_wrong_device_offsets_are_reported():
    c = Case([40, 30], 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for seg in (-1, 32):
        status.zero_()
        c.cu_dev = torch.from_numpy(c.cu).cuda()
        c.fwd(device_status=status, segment_tokens=seg)
        c.bwd(device_status=status, segment_tokens=seg)
        assert int(status) == 0
        for wrong in ([0, 41, 70], [0, 40, 7000], [-5, 40, 70], [0, 400, 70], [70, 0, 3]):
            c.cu_dev = torch.tensor(wrong, dtype=torch.int32, device="cuda")
            for call in (c.fwd, c.bwd):
                status.zero_()
                call(device_status=status, segment_tokens=seg)
                assert int(status) == gdn.binding.GDN_DEVICE_CU_SEQLENS_MISMATCH


def test_autograd_streams_and_graphs():
    c = Case([33, 0, 100], 48, 16, 2, wider=8)
    fields = ("x", "dt", "A_log", "B", "C", "D", "z", "bias", "h0")
    leaf = {n: getattr(c, n).detach().clone().requires_grad_() for n in fields}
    y, ht = gdn.selective_scan(*(leaf[n][None] if n in "xdtBC" else leaf[n] for n in fields[:5]), D=leaf["D"],
                               z=leaf["z"][None], dt_bias=leaf["bias"], initial_state=leaf["h0"],
                               output_final_state=True, cu_seqlens=c.cu_dev, cu_seqlens_cpu=c.cu)
    torch.autograd.backward([y, ht], [c.dy[None], c.dht])
    want = c.bwd()
    for n, g in zip(fields, ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")):
        assert torch.equal(leaf[n].grad, want[g]), n
    assert torch.equal(y[0], c.fwd()[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = c.bwd(segment_tokens=32)
    torch.cuda.synchronize()
    split = c.bwd(segment_tokens=32)
    assert all(torch.equal(again[k], split[k]) for k in split)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*c.fwd(segment_tokens=32), *c.bwd(segment_tokens=32).values())
    for t in (c.x, c.dt, c.B, c.dy):
        t.copy_(torch.randn_like(t))
    graph.replay()
    for a, b in zip(got, (*c.fwd(segment_tokens=32), *c.bwd(segment_tokens=32).values())):
        assert torch.equal(a, b)
