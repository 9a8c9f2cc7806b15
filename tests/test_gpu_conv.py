"""The short causal convolution on the GPU against its 64-bit definition: widths, types, packs with
empty and short sequences, states, pools, steps, gradients, strided rows, streams and graphs."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import mixer_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, lens, C, W=4, dtype=BF, bias=True, silu=True, seed=0, wider=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rn = lambda *s, t=dtype: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.cu_dev = torch.from_numpy(self.cu).cuda()
        T, N = int(self.cu[-1]), len(lens)
        self.x = rn(T, C + wider)[:, wider // 2:wider // 2 + C]
        self.w, self.bias = rn(C, W, t=F32), rn(C, t=F32) if bias else None
        self.h0, self.dht, self.dy = rn(N, C, W - 1), rn(N, C, W - 1), rn(T, C)
        self.act, self.silu, self.t = "silu" if silu else None, silu, dtype

    def kw(self, **more):
        return dict(bias=self.bias, activation=self.act, **more)

    def fwd(self, **kw):
        return gdn.short_conv_fwd(self.x, self.w, self.cu, self.cu_dev, **self.kw(initial_state=self.h0, **kw))

    def bwd(self, **kw):
        return gdn.short_conv_bwd(self.x, self.w, self.dy, self.cu, self.cu_dev,
                                  **self.kw(initial_state=self.h0, d_final_state=self.dht, **kw))

    def reference(self, h0=True, grads=False):
        return ref.conv(self.x, self.w, self.cu, self.bias, self.silu, self.h0 if h0 else None,
                        self.dy if grads else None, self.dht if grads else None)

    def check_fwd(self, y, ht, h0=True):
        (want, off), last, _, _ = self.reference(h0)
        ref.check("y", y, want, off + ref.HALF[self.t] * want.abs() + 1e-30)
        if ht is not None:
            assert torch.equal(ht.double(), last)


SHAPES = [([5], 8, 4), ([1], 1, 2), ([0, 1, 2, 3, 0, 4, 70], 24, 4), ([64, 65, 1, 130], 128, 3), ([3, 0], 7, 4),
          ([300, 17], 1031, 2), ([1] * 40, 16, 4), ([200], 2056, 4)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens, C, W", SHAPES)
def test_forward_and_gradient(lens, C, W, dtype):
    for bias, silu in ((True, True), (False, False)):
        c = Case(lens, C, W, dtype, bias, silu, seed=len(lens))
        c.check_fwd(*c.fwd())
        _, _, g, m = c.reference(grads=True)
        got = c.bwd()
        assert (got["dbias"] is None) == (not bias)
        for name, key, t in (("dx", "dx", dtype), ("dw", "dw", F32), ("dbias", "db", F32), ("dh0", "dh0", dtype)):
            if got[name] is not None:
                ref.check(name, got[name], g[key], m[key] + ref.HALF[t] * g[key].abs() + 1e-30)


def test_without_states():
    c = Case([3, 0, 50], 40)
    y, none = gdn.short_conv_fwd(c.x, c.w, c.cu, c.cu_dev, **c.kw(output_final_state=False))
    assert none is None
    c.check_fwd(y, None, h0=False)
    got = gdn.short_conv_bwd(c.x, c.w, c.dy, c.cu, c.cu_dev, **c.kw(want_dh0=False))
    _, _, g, m = ref.conv(c.x, c.w, c.cu, c.bias, True, None, c.dy, None)
    assert got["dh0"] is None
    ref.check("dx", got["dx"], g["dx"], m["dx"] + ref.HALF[BF] * g["dx"].abs() + 1e-30)


@pytest.mark.parametrize("C, wider", [(64, 64), (64, 3), (33, 31)])
def test_rows_that_lie_apart(C, wider):
    c, d = Case([70, 9], C, wider=wider), Case([70, 9], C, wider=wider)
    d.x = d.x.contiguous()
    for a, b in zip((*c.fwd(), *c.bwd().values()), (*d.fwd(), *d.bwd().values())):
        assert torch.equal(a, b)
    pool = torch.randn(80, C, 3, device="cuda").to(BF)
    idx = torch.arange(79, dtype=torch.int32, device="cuda") + 1
    p, q = pool.clone(), pool.clone()
    assert torch.equal(gdn.short_conv_step(c.x, c.w, p, idx), gdn.short_conv_step(d.x, d.w, q, idx))
    assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens, C, W", [([1, 65, 0, 2], 24, 4), ([7], 9, 3)])
def test_paged_prefill_is_the_forward_over_slots(lens, C, W, dtype):
    c = Case(lens, C, W, dtype)
    N = len(lens)
    pool = torch.randn(N + 3, C, W - 1, device="cuda").to(dtype)
    idx = torch.arange(N, 0, -1, dtype=torch.int32, device="cuda")
    resume = torch.ones(N, dtype=torch.int32, device="cuda")
    resume[0] = 0
    before = pool.clone()
    y = gdn.short_conv_prefill_paged(c.x, c.w, c.cu, c.cu_dev, pool, idx, resume, **c.kw())
    c.h0 = before[idx.long()].clone()
    c.h0[0] = 0
    want, last = c.fwd()
    assert torch.equal(y, want) and torch.equal(pool[idx.long()], last)
    rest = [0, *range(N + 1, N + 3)]
    assert torch.equal(pool[rest], before[rest])


def test_slots_that_are_none_or_outside():
    c = Case([4, 5, 6], 16)
    pool = torch.randn(3, 16, 3, device="cuda").to(BF)
    before, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda")
    y = gdn.short_conv_prefill_paged(c.x, c.w, c.cu, c.cu_dev, pool, idx, device_status=status, **c.kw())
    c.h0[:2], c.h0[2] = 0, before[2]
    want, last = c.fwd()
    assert torch.equal(y, want) and int(status) == 1
    assert torch.equal(pool[:2], before[:2]) and torch.equal(pool[2], last[2])
    status.zero_()
    x = torch.randn(4, 16, device="cuda").to(BF)
    pool, before = before.clone(), before
    idx = torch.tensor([-1, 1, 3, 0], dtype=torch.int32, device="cuda")
    y = gdn.short_conv_step(x, c.w, pool, idx, device_status=status, **c.kw())
    assert int(status) == 1 and not y[[0, 2, 3]].any() and y[1].any()
    assert torch.equal(pool[[0, 2]], before[[0, 2]]) and torch.equal(pool[1, :, 2], x[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C, W", [(8, 4), (1, 2), (2056, 3), (1031, 4)])
def test_steps_are_the_forward(C, W, dtype):
    c = Case([6, 6, 6], C, W, dtype)
    pool = torch.zeros(5, C, W - 1, device="cuda", dtype=dtype)
    idx = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    pool[idx.long()] = c.h0
    x = c.x.reshape(3, 6, C)
    y = torch.stack([gdn.short_conv_step(x[:, t].contiguous(), c.w, pool, idx, **c.kw()) for t in range(6)], 1)
    c.check_fwd(y.reshape(18, C), pool[idx.long()])


def test_no_tokens_and_no_rows():
    c = Case([0, 0], 16)
    y, ht = c.fwd()
    assert y.shape == (0, 16) and torch.equal(ht, c.h0)
    got = c.bwd()
    assert torch.equal(got["dh0"], c.dht) and not got["dw"].any() and not got["dbias"].any()
    pool = torch.randn(2, 16, 3, device="cuda").to(BF)
    assert gdn.short_conv_step(c.x, c.w, pool, torch.zeros(0, dtype=torch.int32, device="cuda")).shape == (0, 16)


def test_infinities_stay_in_their_window():
    c = Case([40, 30], 16, silu=False)
    c.x[10, 3] = float("inf")
    c.x[69, 5] = float("nan")
    y, ht = c.fwd()
    bad = ~torch.isfinite(y)
    assert bad[10:14, 3].all() and bad[69, 5] and int(bad.sum()) == 5
    assert torch.isnan(ht[1, 5, 2])


def test_wrong_device_offsets_are_reported():
    c = Case([40, 30], 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.fwd(device_status=status)
    c.bwd(device_status=status)
    assert int(status) == 0
    for wrong in ([0, 41, 70], [0, 40, 7000], [-5, 40, 70], [0, 400, 70]):
        c.cu_dev = torch.tensor(wrong, dtype=torch.int32, device="cuda")
        for call in (c.fwd, c.bwd):
            status.zero_()
            call(device_status=status)
            assert int(status) == gdn.binding.GDN_DEVICE_CU_SEQLENS_MISMATCH


def test_autograd_streams_and_graphs():
    c = Case([33, 0, 100], 48, wider=16)
    x, w, b, h0 = (t.detach().clone().requires_grad_() for t in (c.x, c.w, c.bias, c.h0))
    kw = dict(initial_state=h0, output_final_state=True, cu_seqlens=c.cu_dev, cu_seqlens_cpu=c.cu)
    y, ht = gdn.short_conv(x[None], w, b, **kw)
    torch.autograd.backward([y, ht], [c.dy[None], c.dht])
    want = c.bwd()
    for a, b_ in ((x.grad, "dx"), (w.grad, "dw"), (b.grad, "dbias"), (h0.grad, "dh0")):
        assert torch.equal(a, want[b_])
    assert torch.equal(y[0], c.fwd()[0]) and torch.equal(ht, c.fwd()[1])
    # a loss of the final state alone, weights in bf16
    w16 = c.w.to(BF).requires_grad_()
    _, ht = gdn.short_conv(c.x, w16, None, **dict(kw, initial_state=None))
    x2 = c.x.detach().clone().requires_grad_()
    gdn.short_conv(x2, w16, None, **dict(kw, initial_state=None))[1].float().sum().backward()
    assert not w16.grad.any() and float(x2.grad.sum()) == 3 * 48 * 2
    # another stream, and a graph replayed with other inputs
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = c.bwd()
    torch.cuda.synchronize()
    assert all(torch.equal(again[k], want[k]) for k in want)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*c.fwd(), *c.bwd(workspace=ws).values())
    c.x.copy_(torch.randn_like(c.x))
    graph.replay()
    for a, b_ in zip(got, (*c.fwd(), *c.bwd().values())):
        assert torch.equal(a, b_)
