"""Decay-only linear attention on the GPU against its 64-bit definition: packs of every
length, shared key heads, decays from none to total, the pool forms, gradients, refusals."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import linear_reference as ref

pytestmark = pytest.mark.gpu

DECAYS = [-0.02, 0.0, -6.0, -0.5, -1e-6, -100.0, float("-inf"), -0.003]


def _bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().to(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, lens, H, HV, seed=0, states=True):
        rng = np.random.default_rng([seed, 77])
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        T, N = int(self.cu[-1]), len(lens)
        self.cu_dev = torch.from_numpy(self.cu).cuda()
        self.q, self.k = (_bf(rng.standard_normal((T, H, 128))) for _ in range(2))
        self.v, self.do = (_bf(rng.standard_normal((T, HV, 128))) for _ in range(2))
        self.g = torch.tensor((DECAYS * HV)[seed:seed + HV], dtype=torch.float32).cuda()
        mk = lambda: torch.from_numpy(rng.standard_normal((N, HV, 128, 128)).astype(np.float32)).cuda()  # noqa: E731
        self.h0, self.dht = (mk(), mk()) if states else (None, None)

    def host(self, mag=False):
        f = (lambda t: None if t is None else np.abs(_f64(t))) if mag else (
            lambda t: None if t is None else _f64(t))
        return (f(self.q), f(self.k), f(self.v), _f64(self.g), self.cu)

    def fwd(self, **kw):
        return gdn.linear_attn_fwd(self.q, self.k, self.v, self.g, self.cu, self.cu_dev,
                                   initial_state=self.h0, **kw)

    def bwd(self, **kw):
        return gdn.linear_attn_bwd(self.q, self.k, self.v, self.g, self.do, self.cu, self.cu_dev,
                                   initial_state=self.h0, d_final_state=self.dht, **kw)

    def ref_fwd(self):
        h = None if self.h0 is None else _f64(self.h0)
        return ref.forward(*self.host(), h), ref.forward(*self.host(True), None if h is None else np.abs(h))

    def ref_bwd(self):
        h, d = (None, None) if self.h0 is None else (_f64(self.h0), _f64(self.dht))
        a = ref.backward(*self.host(), _f64(self.do), h, d)
        ab = (None, None) if h is None else (np.abs(h), np.abs(d))
        return a, ref.backward(*self.host(True), np.abs(_f64(self.do)), *ab)

    def check_fwd(self, o, ht):
        (ro, rh), (mo, mh) = self.ref_fwd()
        ref.check("o", o, ro, ref.out_bound(ro, mo))
        if ht is not None:
            ref.check("final_state", ht, rh, ref.state_bound(mh))

    def check_bwd(self, gr):
        r, m = self.ref_bwd()
        for n in ("dq", "dk", "dv"):
            ref.check(n, gr[n], r[n], ref.out_bound(r[n], m[n]))
        if gr["dh0"] is not None:
            ref.check("dh0", gr["dh0"], r["dh0"], ref.state_bound(m["dh0"]))


PACKS = [([1], 1, 1), ([63], 1, 2), ([64], 2, 2), ([65], 1, 1), ([127], 1, 3), ([128], 2, 4), ([129], 1, 1),
         ([255], 1, 1), ([257, 1, 64], 1, 2), ([0, 5, 0, 130, 0], 2, 4), ([300, 128, 77], 1, 4), ([40] * 9, 2, 2),
         ([700], 1, 1), ([31, 513], 1, 5)]


@pytest.mark.parametrize("i", range(len(PACKS)))
@pytest.mark.parametrize("states", [True, False])
def test_forward(i, states):
    c = Case(*PACKS[i], seed=i % len(DECAYS), states=states)
    c.check_fwd(*c.fwd())
    o, none = c.fwd(output_final_state=False)
    assert none is None and torch.equal(o, c.fwd()[0])


@pytest.mark.parametrize("i", range(len(PACKS)))
@pytest.mark.parametrize("states", [True, False])
def test_backward(i, states):
    c = Case(*PACKS[i], seed=(i + 3) % len(DECAYS), states=states)
    gr = c.bwd()
    c.check_bwd(gr)
    assert c.bwd(want_dh0=False)["dh0"] is None


SPLITS = [([700], 1, 1, 1), ([700, 0, 129, 1], 1, 2, 2), ([300, 900], 2, 2, 3), ([640], 1, 3, 4), ([385], 1, 4, 1)]


@pytest.mark.parametrize("lens, H, HV, seg", SPLITS)
def test_split_scans(lens, H, HV, seg):
    c = Case(lens, H, HV, seed=HV)
    c.check_fwd(*c.fwd(scan_segment_chunks=seg))
    c.check_bwd(c.bwd(scan_segment_chunks=seg))
    # without splitting, the same values to the same bounds (checked above): outputs of the
    # first segment are the same bits
    whole = c.fwd(scan_segment_chunks=-1)[0]
    assert torch.equal(c.fwd(scan_segment_chunks=seg)[0][:min(lens[0], 128 * seg)], whole[:min(lens[0], 128 * seg)])


def test_the_plan_splits_a_long_sequence():
    c = Case([5000, 2100], 1, 2)
    n = [gdn.gdn_linear_attn_workspace_bytes(
        gdn.make_problem(c.cu, 1, 2, cu_dev_ptr=c.cu_dev.data_ptr(), scan_segment_chunks=x)[0], 0) for x in (0, -1)]
    assert n[0] > n[1]
    c.check_fwd(*c.fwd())
    c.check_bwd(c.bwd())


def test_split_paged_prefill_starts_from_the_slot_it_ends_in():
    c = Case([900, 260], 1, 2)
    pool = torch.randn(3, 2, 128, 128, device="cuda")
    c.h0 = pool[1:].transpose(2, 3).contiguous()
    want, ht = c.fwd(scan_segment_chunks=2)
    idx = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    o = gdn.linear_attn_prefill_paged(c.q, c.k, c.v, c.g, c.cu, c.cu_dev, pool, idx, scan_segment_chunks=2)
    assert torch.equal(o, want) and torch.equal(pool[1:].transpose(2, 3), ht)


def test_many_sequences():
    c = Case([3, 0, 130] * 50, 1, 1)
    c.check_fwd(*c.fwd())
    c.check_bwd(c.bwd())


def test_eight_value_heads_to_a_key_head():
    c = Case([200], 1, 8)
    c.check_fwd(*c.fwd())
    c.check_bwd(c.bwd())
    c = Case([150], 1, 9)
    c.check_bwd(c.bwd())


def test_scale_argument():
    c = Case([150], 1, 1, seed=0)
    (ro, rh), (mo, mh) = c.ref_fwd()
    o, ht = c.fwd(scale=0.5)
    f = 0.5 * 128 ** 0.5
    ref.check("o", o, f * ro, ref.out_bound(f * ro, f * mo))
    ref.check("final_state", ht, rh, ref.state_bound(mh))


def test_slow_decay_over_a_long_sequence():
    # the per-chunk factor must hold more than fp32: 2^-25 of it would grow over the chunks
    T, g = 16384, -1e-5
    c = Case([T], 1, 1)
    c.g.fill_(g)
    lam = np.exp(np.float64(np.float32(g)))
    w = lam ** np.arange(T - 1, -1, -1, dtype=np.float64)
    k, v, h0 = _f64(c.k)[:, 0], _f64(c.v)[:, 0], _f64(c.h0)[0, 0]
    want = (k * w[:, None]).T @ v + lam ** T * h0
    mag = (np.abs(k) * w[:, None]).T @ np.abs(v) + lam ** T * np.abs(h0)
    ref.check("final_state", c.fwd()[1][0, 0], want, ref.state_bound(mag))


def test_empty_pack_passes_the_state():
    c = Case([0, 0], 1, 2)
    o, ht = c.fwd()
    assert o.shape == (0, 2, 128) and torch.equal(ht, c.h0)
    assert torch.equal(c.bwd()["dh0"], c.dht)
    c = Case([0], 1, 2, states=False)
    assert not c.fwd()[1].any() and not c.bwd()["dh0"].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_are_untouched_by_bad_values(bad):
    c = Case([70, 130, 20], 1, 2)
    clean, gr = c.fwd(), c.bwd()
    for x in (c.q, c.k, c.v, c.do):
        x[70:200] = bad
    c.h0[1] = bad
    c.dht[1] = bad
    o, ht = c.fwd()
    bw = c.bwd()
    for a, b in ((o, clean[0]), (bw["dq"], gr["dq"]), (bw["dk"], gr["dk"]), (bw["dv"], gr["dv"])):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[200:], b[200:])
    for a, b in ((ht, clean[1]), (bw["dh0"], gr["dh0"])):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_runs_are_bit_identical_on_any_stream():
    c = Case([257, 600, 31], 2, 4)
    one, g1 = c.fwd(), c.bwd()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two, g2 = c.fwd(), c.bwd()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert all(torch.equal(g1[n], g2[n]) for n in g1)


def test_paged_prefill_is_the_forward_over_slots():
    c = Case([130, 1, 0, 300, 40], 2, 4)
    pool = torch.randn(8, 4, 128, 128, device="cuda")
    before = pool.clone()
    idx = torch.tensor([3, 5, 7, 0, 9], dtype=torch.int32, device="cuda")  # 0: none; 9: out of range
    resume = torch.tensor([1, 0, 1, 1, 1], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = gdn.linear_attn_prefill_paged(c.q, c.k, c.v, c.g, c.cu, c.cu_dev, pool, idx, resume,
                                      device_status=status)
    c.h0 = torch.zeros(5, 4, 128, 128, device="cuda")
    c.h0[0] = before[3].transpose(1, 2)
    c.h0[2] = before[7].transpose(1, 2)
    want, ht = c.fwd()
    assert torch.equal(o, want) and int(status) == 1
    for n, slot in ((0, 3), (1, 5), (2, 7)):
        assert torch.equal(pool[slot], ht[n].transpose(1, 2))
    for slot in (0, 1, 2, 4, 6):
        assert torch.equal(pool[slot], before[slot])


@pytest.mark.parametrize("B, H, HV", [(1, 1, 1), (3, 2, 2), (7, 2, 6), (33, 4, 8)])
def test_step(B, H, HV):
    rng = np.random.default_rng(B)
    q, k = (_bf(rng.standard_normal((B, H, 128))) for _ in range(2))
    v = _bf(rng.standard_normal((B, HV, 128)))
    g = torch.tensor((DECAYS * 2)[:HV], dtype=torch.float32, device="cuda")
    pool = torch.from_numpy(rng.standard_normal((B + 3, HV, 128, 128)).astype(np.float32)).cuda()
    before = _f64(pool)
    idx = torch.arange(B, 0, -1, dtype=torch.int32, device="cuda")
    if B > 2:
        idx[1], idx[2] = -1, B + 3  # null, out of range
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = gdn.linear_attn_step(q, k, v, g, pool, idx, device_status=status)
    assert int(status) == (1 if B > 2 else 0)
    after = before.copy()
    for b, slot in enumerate(idx.tolist()):
        if not 0 < slot < B + 3:
            assert not o[b].any()
            continue
        one = lambda f: ref.forward(f(_f64(q[b:b + 1])), f(_f64(k[b:b + 1])), f(_f64(v[b:b + 1])), _f64(g), [0, 1],  # noqa: E731
                                    f(before[slot:slot + 1].transpose(0, 1, 3, 2)))
        (ro, rh), (mo, mh) = one(lambda x: x), one(np.abs)
        ref.check("o", o[b:b + 1], ro, ref.out_bound(ro, mo))
        ref.check("slot", pool[slot:slot + 1].transpose(2, 3), rh, ref.state_bound(mh))
        after[slot] = _f64(pool[slot])
    assert np.array_equal(after, _f64(pool))  # no other slot changed


def test_step_continues_a_prefill():
    c = Case([129], 2, 4, states=False)
    whole, ht = c.fwd()
    pool = torch.zeros(2, 4, 128, 128, device="cuda")
    idx = torch.ones(1, dtype=torch.int32, device="cuda")
    cu = np.array([0, 128], np.int32)
    gdn.linear_attn_prefill_paged(c.q[:128], c.k[:128], c.v[:128], c.g, cu, torch.from_numpy(cu).cuda(), pool, idx)
    o = gdn.linear_attn_step(c.q[128:], c.k[128:], c.v[128:], c.g, pool, idx)
    (ro, rh), (mo, mh) = c.ref_fwd()
    ref.check("o", o, ro[128:], ref.out_bound(ro, mo)[128:])
    ref.check("state", pool[1:].transpose(2, 3), rh, ref.state_bound(mh))


def test_many_steps_of_a_slow_decay():
    # lam in fp32 would be off by up to 2^-25 each step, 2^-15 after 1024
    n, g = 1024, -3e-4
    rng = np.random.default_rng(3)
    q, k, v = (_bf(rng.standard_normal((n, 1, 128))) for _ in range(3))
    gd = torch.full((1,), g, device="cuda")
    pool = torch.randn(2, 1, 128, 128, device="cuda")
    s0 = _f64(pool[1, 0])
    idx = torch.ones(1, dtype=torch.int32, device="cuda")
    for t in range(n):
        gdn.linear_attn_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], gd, pool, idx)
    w = np.exp(np.float64(np.float32(g)) * np.arange(n, -1, -1))
    kk, vv = _f64(k)[:, 0], _f64(v)[:, 0]
    want = (vv * w[1:, None]).T @ kk + w[0] * s0
    mag = (np.abs(vv) * w[1:, None]).T @ np.abs(kk) + w[0] * np.abs(s0)
    ref.check("slot", pool[1, 0], want, ref.state_bound(mag))


def test_autograd():
    c = Case([100, 61], 2, 4)
    q, k, v = (x.clone().requires_grad_() for x in (c.q, c.k, c.v))
    h0 = c.h0.clone().requires_grad_()
    o, ht = gdn.linear_attention(q[None], k[None], v[None], c.g, initial_state=h0, output_final_state=True,
                                 cu_seqlens=c.cu_dev, cu_seqlens_cpu=c.cu)
    torch.autograd.backward([o, ht], [c.do[None], c.dht])
    gr = c.bwd()
    for t, n in ((q, "dq"), (k, "dk"), (v, "dv"), (h0, "dh0")):
        assert torch.equal(t.grad, gr[n])
    with pytest.raises(ValueError):
        gdn.linear_attention(q, k, v, c.g.clone().requires_grad_())


def test_bounds_checked_build():
    from chunked_gated_delta_06_gb300 import binding, build
    c = Case([130, 1, 300], 2, 4)
    want, gr = c.fwd(), c.bwd()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with binding.use_library(build.build(checked=True)):
        o, ht = c.fwd(device_status=status)
        ck = c.bwd(device_status=status)
    assert int(status) == 0 and torch.equal(o, want[0]) and torch.equal(ht, want[1])
    assert all(torch.equal(ck[n], gr[n]) for n in gr)


def test_device_offsets_that_disagree_are_flagged():
    c = Case([64, 64], 1, 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.fwd(device_status=status)
    assert int(status) == 0
    c.cu_dev[1] = 100
    c.fwd(device_status=status)
    assert int(status) == gdn.binding.GDN_DEVICE_CU_SEQLENS_MISMATCH


def test_python_calls_refuse_what_the_kernels_cannot_read():
    c = Case([64], 2, 4)
    args = lambda **kw: [kw.get(n, getattr(c, n)) for n in ("q", "k", "v", "g", "cu", "cu_dev")]  # noqa: E731
    with pytest.raises(TypeError):
        gdn.linear_attn_fwd(*args(q=c.q.float()))
    for bad in (dict(k=c.k[:, :1]), dict(v=c.v.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(g=c.g[:2]), dict(q=c.q.cpu()), dict(cu=c.cu[:1])):
        with pytest.raises(ValueError):
            gdn.linear_attn_fwd(*args(**bad))
    with pytest.raises(gdn.GdnError):
        gdn.linear_attn_fwd(c.q[:, :, :64].contiguous(), c.k[:, :, :64].contiguous(), c.v, c.g, c.cu, c.cu_dev)
    with pytest.raises(ValueError):
        gdn.linear_attn_bwd(*args()[:4], c.do[:10], c.cu, c.cu_dev)


# Sequences of one chunk: the second bf16 parts leave 2^-16 of each term, the fp32 sums at most
# 2^-12, and the output is rounded once.  (One or three value heads a key head: no exchange.)
@pytest.mark.parametrize("lens, H, HV", [([1], 1, 1), ([2, 1, 0, 7], 2, 2), ([128], 1, 1), ([40] * 3, 1, 3),
                                         ([127, 65], 1, 1)])
@pytest.mark.parametrize("states", [True, False])
def test_one_chunk_outputs(lens, H, HV, states):
    c = Case(lens, H, HV, seed=3, states=states)
    bound = lambda r, m: 2.0 ** -12 * m + 2.0 ** -7.9 * np.abs(r) + 1e-30  # noqa: E731
    (ro, _), (mo, _) = c.ref_fwd()
    ref.check("o", c.fwd()[0], ro, bound(ro, mo))
    (r, m), gr = c.ref_bwd(), c.bwd()
    for n in ("dq", "dk", "dv"):
        ref.check(n, gr[n], r[n], bound(r[n], m[n]))


@pytest.mark.parametrize("lens", [[5], [130]])
def test_infinite_state_stays_in_its_column(lens):
    c = Case(lens, 1, 1, seed=0)
    c.h0[0, 0, 3, 7] = float("inf")   # [K, V]
    o, _ = c.fwd()
    assert torch.isinf(o[:, :, 7]).all()
    o[:, :, 7] = 0
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("H, HV", [(1, 1), (1, 2), (1, 4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_between_sequences_of_one_chunk(H, HV, bad):
    c = Case([70, 20, 128, 33], H, HV)
    clean, gr = c.fwd(), c.bwd()
    for x in (c.q, c.k, c.v, c.do):
        x[70:90] = bad
    c.h0[1] = bad
    c.dht[1] = bad
    o, ht = c.fwd()
    bw = c.bwd()
    rest = [i for i in range(251) if not 70 <= i < 90]
    for a, b in ((o, clean[0]), (bw["dq"], gr["dq"]), (bw["dk"], gr["dk"]), (bw["dv"], gr["dv"])):
        assert torch.equal(a[rest], b[rest])
    for a, b in ((ht, clean[1]), (bw["dh0"], gr["dh0"])):
        assert torch.equal(a[[0, 2, 3]], b[[0, 2, 3]])


def test_many_sequences_of_one_chunk():
    c = Case([3, 0, 120, 17] * 40, 1, 2)
    c.check_fwd(*c.fwd())
    c.check_bwd(c.bwd())


# Pairs whose scans of different lengths share the SMs, many times over: the same bits.
def test_backward_of_pairs_repeats():
    c = Case([300, 1, 0, 130, 257, 128, 40], 2, 4)
    first = c.bwd()
    for _ in range(30):
        again = c.bwd()
        assert all(torch.equal(first[n], again[n]) for n in first)
