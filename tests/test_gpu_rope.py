"""Rotary positions on the GPU against the 64-bit rotation: layouts, parts of the head, far
positions, the gradient, in place."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_06_gb300 as gdn

import linear_reference as ref

pytestmark = pytest.mark.gpu


def _inputs(T, Hq, Hk, D, rot, seed=0, positions=None, **freq):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q, k = (torch.randn(T, h, D, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hk))
    pos = (torch.randint(0, 131072, (T,), generator=g, device="cuda", dtype=torch.int32) if positions is None
           else torch.tensor(positions, dtype=torch.int32, device="cuda"))
    return q, k, pos, gdn.rope_frequencies(rot, **freq)


def _check(x, y, pos, freq, layout, m=1.0, backward=False):
    xd = x.double().cpu().numpy()
    want = ref.rope(xd, pos.cpu().numpy(), freq.cpu().numpy(), layout, m, backward)
    # one rounding to bf16 (half an ulp: 2^-8), products of fp32 factors, and an angle good to 2^-20 turns
    # on the larger of the pair's elements (bounded by the head's largest)
    big = np.abs(xd).max(-1, keepdims=True)
    ref.check("rope", y, want, 2.0 ** -7.9 * np.abs(want) + abs(m) * 2.0 ** -16 * big)
    rot = 2 * freq.shape[1]
    assert torch.equal(x[..., rot:], y[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T, Hq, Hk, D, rot", [(1, 1, 1, 128, 128), (7, 4, 1, 128, 64), (33, 2, 2, 96, 24), (5, 3, 1, 64, 2),
                                               (17, 2, 1, 256, 64), (3, 1, 1, 6, 4), (300, 16, 4, 80, 40)])
def test_rotation(layout, backward, T, Hq, Hk, D, rot):
    q, k, pos, freq = _inputs(T, Hq, Hk, D, rot)
    qo, ko = gdn.rope(q, k, pos, freq, layout=layout, backward=backward)
    _check(q, qo, pos, freq, layout, backward=backward)
    _check(k, ko, pos, freq, layout, backward=backward)
    # in place, and without k, the same bits
    q2, k2 = q.clone(), k.clone()
    a, b = gdn.rope(q2, k2, pos, freq, layout=layout, backward=backward, inplace=True)
    assert a is q2 and b is k2 and torch.equal(q2, qo) and torch.equal(k2, ko)
    alone, none = gdn.rope(q, None, pos, freq, layout=layout, backward=backward)
    assert none is None and torch.equal(alone, qo)


def test_far_and_negative_positions():
    pos = [0, 1, -1, -70000, 65535, 65536, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)]
    q, k, pos, freq = _inputs(len(pos), 2, 1, 128, 128, positions=pos)
    qo, ko = gdn.rope(q, k, pos, freq)
    _check(q, qo, pos, freq, "half")
    assert torch.equal(qo[0], q[0])


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=8.0), dict(scaling="parts", factor=4.0, trained_len=4096)])
def test_scaled_frequencies(kw):
    q, k, pos, freq = _inputs(65, 2, 2, 128, 128, **kw)
    qo, ko = gdn.rope(q, k, pos, freq, mscale=1.1386)
    _check(q, qo, pos, freq, "half", 1.1386)
    _check(k, ko, pos, freq, "half", 1.1386)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_is_the_transpose(layout):
    q, k, pos, freq = _inputs(9, 2, 1, 128, 64)
    x, y = q.clone().requires_grad_(), k.clone().requires_grad_()
    qo, ko = gdn.rotary(x, y, pos, freq, layout, 1.25)
    dq, dk = torch.randn_like(qo), torch.randn_like(ko)
    torch.autograd.backward([qo, ko], [dq, dk])
    _check(dq, x.grad, pos, freq, layout, 1.25, True)
    _check(dk, y.grad, pos, freq, layout, 1.25, True)
    # <rope(x), dq> = <x, rope_backward(dq)>, in 64 bits
    f = lambda t, b: ref.rope(t.detach().double().cpu().numpy(), pos.cpu().numpy(), freq.cpu().numpy(), layout, 1.25, b)  # noqa: E731
    a = (f(q, False) * dq.double().cpu().numpy()).sum()
    b = (q.double().cpu().numpy() * f(dq, True)).sum()
    assert abs(a - b) <= 1e-9 * (1 + abs(a))


def test_no_tokens_and_refusals():
    q, k, pos, freq = _inputs(4, 2, 1, 128, 64)
    e, n = gdn.rope(q[:0], k[:0], pos[:0], freq)
    assert e.shape == (0, 2, 128) and n.shape == (0, 1, 128)
    with pytest.raises(TypeError):
        gdn.rope(q.float(), k, pos, freq)
    with pytest.raises(TypeError):
        gdn.rope(q, k, pos.long(), freq)
    for bad in (dict(k=k[:3]), dict(q=q[:, :, ::2]), dict(pos=pos[:2]), dict(freq=freq[:1])):
        a = dict(q=q, k=k, pos=pos, freq=freq)
        a.update(bad)
        with pytest.raises(ValueError):
            gdn.rope(a["q"], a["k"], a["pos"], a["freq"])
    with pytest.raises(gdn.GdnError):
        gdn.rope(q, k, pos, torch.zeros(2, 65, device="cuda"))
    with pytest.raises(KeyError):
        gdn.rope(q, k, pos, freq, layout="other")


def test_the_most_tokens():
    # 2^31 - 1 tokens of one pair: the number of blocks does not pass 32 bits on its way (17 GB)
    T = 2 ** 31 - 1
    q = torch.empty(T, 1, 2, device="cuda", dtype=torch.bfloat16)
    pos = torch.empty(T, device="cuda", dtype=torch.int32)
    freq = gdn.rope_frequencies(2)
    rows = torch.tensor([0, 1, 2 ** 30 + 1, T - 2, T - 1], device="cuda")
    q[rows] = torch.randn(5, 1, 2, device="cuda").to(torch.bfloat16)
    pos[rows] = torch.tensor([3, 70000, -5, 11, 2 ** 31 - 1], device="cuda", dtype=torch.int32)
    x = q[rows]
    gdn.rope(q, None, pos, freq, inplace=True)
    _check(x, q[rows], pos[rows], freq, "half")
