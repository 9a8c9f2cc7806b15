"""Decay-only linear attention at the edges of the number range: scales, columns of very different
size, infinities in the states, against the 64-bit definition."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import linear_reference as ref
from test_gpu_linear import Case, _f64

pytestmark = pytest.mark.gpu


def _check_bwd(c, scale):
    """The backward at a scale against the reference, to the bounds of the other tests."""
    gr = c.bwd(scale=scale)
    h, d = (None, None) if c.h0 is None else (_f64(c.h0), _f64(c.dht))
    ab = (None, None) if h is None else (np.abs(h), np.abs(d))
    r = ref.backward(*c.host(), _f64(c.do), h, d, scale=scale)
    m = ref.backward(*c.host(True), np.abs(_f64(c.do)), *ab, scale=scale)
    for n in ("dq", "dk", "dv"):
        ref.check(n, gr[n], r[n], ref.out_bound(r[n], m[n]))
    ref.check("dh0", gr["dh0"], r["dh0"], ref.state_bound(m["dh0"]))


# Tokens without a gradient (a loss mask, padding) give rows of zeros in the sum of a pair.
@pytest.mark.parametrize("lens", [[70], [300, 40]])
@pytest.mark.parametrize("HV", [1, 2, 4])
@pytest.mark.parametrize("scale", [1.0, 4.0, 11.3])
def test_backward_of_masked_tokens_at_any_scale(lens, HV, scale):
    c = Case(lens, 1, HV, seed=3, states=False)
    c.do[::3] = 0
    c.do[40:60] = 0
    c.q[10:20] = 0
    c.h0 = c.dht = None
    _check_bwd(c, scale)


def _columns(name, got, want, bound, bad):
    """Feature `bad` of `got` is infinite wherever the definition has it so, the rest within bounds."""
    got = _f64(got)
    assert not np.isfinite(got[..., bad]).any(), name
    rest = np.arange(got.shape[-1]) != bad
    off = np.abs(got - want)[..., rest] / bound[..., rest]
    assert np.all(off <= 1), "%s: worst %.3g of the bound" % (name, np.nanmax(off))


# An infinite element of a state reaches one feature of a gradient; the features beside it, which
# two value heads add up, keep both heads' parts.
@pytest.mark.parametrize("lens", [[60], [200]])
@pytest.mark.parametrize("HV", [1, 2, 4])
@pytest.mark.parametrize("row, head", [(5, 0), (70, 0), (40, 1), (127, 1)])
def test_backward_beside_an_infinite_state(lens, HV, row, head):
    c = Case(lens, 1, HV, seed=0)
    c.g.fill_(-0.02)
    head = min(head, HV - 1)
    c.h0[0, head, row, 9] = 0
    c.dht[0, head, row, 9] = 0
    r, m = c.ref_bwd()
    c.h0[0, head, row, 9] = float("inf")
    c.dht[0, head, row, 9] = float("-inf")
    gr = c.bwd()
    for n in ("dq", "dk"):
        _columns(n, gr[n][:, 0], r[n][:, 0], ref.out_bound(r[n], m[n])[:, 0], row)
    _columns("dv", gr["dv"][:, head], r["dv"][:, head], ref.out_bound(r["dv"], m["dv"])[:, head], 9)


# A feature of q and k far above its neighbours: every gradient keeps its own precision.
@pytest.mark.parametrize("lens", [[60], [200, 129]])
@pytest.mark.parametrize("HV", [1, 2, 4])
@pytest.mark.parametrize("power", [18, 24, 40])
def test_backward_of_features_of_very_different_size(lens, HV, power):
    c = Case(lens, 1, HV, seed=0)
    for x in (c.q, c.k):
        x[:, :, [7, 90]] *= 2.0 ** power
    c.check_bwd(c.bwd())


INF_DECAYS = [0.0, -1e-6, -0.003, -0.02, -0.3, -0.5, -1.0, -6.0, -100.0]


def _state(name, got, want, bound, at):
    """got[at] has the infinity, every other element is within bounds."""
    got = _f64(got)
    assert got[at] == np.inf, "%s: %r" % (name, got[at])
    got[at] = want[at]
    off = np.abs(got - want) / bound
    assert np.all(off <= 1), "%s: worst %.3g of the bound" % (name, np.nanmax(off))


# An infinite state stays infinite while e^g is not zero, whatever the tail of a chunk's factor.
@pytest.mark.parametrize("lens, seg", [([1], -1), ([130], -1), ([300], -1), ([1300], 2)])
@pytest.mark.parametrize("g", INF_DECAYS)
def test_infinite_state_through_a_scan(lens, seg, g):
    c = Case(lens, 1, 2, seed=0)
    c.g.fill_(g)
    for x in (c.h0, c.dht):
        x[0, 1, 3, 7] = 0
    (_, rh), (_, mh) = c.ref_fwd()
    r, m = c.ref_bwd()
    for x in (c.h0, c.dht):
        x[0, 1, 3, 7] = float("inf")
    _state("final_state", c.fwd(scan_segment_chunks=seg)[1], rh, ref.state_bound(mh), (0, 1, 3, 7))
    _state("dh0", c.bwd(scan_segment_chunks=seg)["dh0"], r["dh0"], ref.state_bound(m["dh0"]), (0, 1, 3, 7))


@pytest.mark.parametrize("g", INF_DECAYS)
def test_infinite_state_through_steps(g):
    rng = np.random.default_rng(4)
    q, k, v = (torch.from_numpy(rng.standard_normal((2, 1, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
               for _ in range(3))
    pool = torch.from_numpy(rng.standard_normal((3, 1, 128, 128)).astype(np.float32)).cuda()
    gd = torch.full((1,), g, device="cuda")
    idx = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    pool[2, 0, 7, 3] = 0   # [V, K]
    before = _f64(pool[1:])[:, 0]
    pool[2, 0, 7, 3] = float("inf")
    o = gdn.linear_attn_step(q, k, v, gd, pool, idx)
    vk = _f64(v)[:, 0, :, None] * _f64(k)[:, 0, None, :]
    lam = np.exp(np.float64(np.float32(g)))
    _state("pool", pool[1:, 0], lam * before + vk, ref.state_bound(lam * np.abs(before) + np.abs(vk)), (1, 7, 3))
    o = _f64(o)[:, 0]
    assert np.isinf(o[1, 7]) and np.isfinite(np.delete(o[1], 7)).all() and np.isfinite(o[0]).all()


# More sequences than a launch carries offsets for: the device's copy is walked, and any difference
# from the host's is reported.
@pytest.mark.parametrize("lens", [[3, 0, 70], [3, 0, 130]])
@pytest.mark.parametrize("wrong", ["shift", "two", "first", "last", "outside", "backwards"])
def test_device_offsets_of_many_sequences(lens, wrong):
    c = Case(lens * 50, 1, 2, states=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = c.fwd(device_status=status), c.bwd(device_status=status)
    assert int(status) == 0
    right, T = c.cu_dev.clone(), int(c.cu[-1])
    at, by = dict(shift=([60], -1), two=([30, 60], -1), first=([0], 1), last=([-1], -1), outside=([75], T),
                  backwards=([75], -T))[wrong]
    c.cu_dev[at] += by
    for call in (c.fwd, c.bwd):
        status.zero_()
        call(device_status=status)
        assert int(status) == gdn.binding.GDN_DEVICE_CU_SEQLENS_MISMATCH
    c.cu_dev.copy_(right)
    again = c.fwd(), c.bwd()
    assert torch.equal(good[0][0], again[0][0]) and all(torch.equal(good[1][n], again[1][n]) for n in again[1])


# An infinite token: its feature of the outputs from there on and of the state is not finite, the
# other features, the tokens of earlier chunks and the other sequences keep their values.
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("g", [0.0, -0.02])
def test_infinite_token_stays_in_its_feature(bad, g):
    c = Case([300, 40], 1, 2, seed=0)
    c.g.fill_(g)
    (ro, rh), (mo, mh) = c.ref_fwd()
    c.v[150, 1, 9] = bad
    o, ht = (_f64(x) for x in c.fwd())
    assert not np.isfinite(o[150:300, 1, 9]).any() and not np.isfinite(ht[0, 1, :, 9]).any()
    for got, want, bound, hit in ((o, ro, ref.out_bound(ro, mo), np.s_[128:300, 1, 9]),
                                  (ht, rh, ref.state_bound(mh), np.s_[0, 1, :, 9])):
        got[hit] = want[hit]
        assert np.all(np.abs(got - want) <= bound)
