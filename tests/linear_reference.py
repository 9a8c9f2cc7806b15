"""64-bit references of the decay-only linear attention and of rotary positions (numpy, from
their definitions), with error bounds for the kernels that compute them."""
import numpy as np

D = 128


def forward(q, k, v, g, cu, h0=None, scale=D ** -0.5):
    """o [T, HV, V], final state [N, HV, K, V] and every token's state, token by token."""
    T, H, _ = q.shape
    HV = v.shape[1]
    r = HV // H
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    q, k = np.repeat(q, r, 1), np.repeat(k, r, 1)
    lam = np.exp(np.asarray(g, np.float64))[:, None, None]
    N = len(cu) - 1
    fin = np.zeros((N, HV, D, D)) if h0 is None else np.array(h0, np.float64)
    o = np.zeros_like(v)
    for n in range(N):
        S = fin[n]
        for t in range(cu[n], cu[n + 1]):
            S *= lam
            S += k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
    return o, fin


def backward(q, k, v, g, cu, do, h0=None, dht=None, scale=D ** -0.5):
    """dq, dk (summed over the value heads of a key head), dv and dh0 by the two recurrences."""
    T, H, _ = q.shape
    HV = v.shape[1]
    r = HV // H
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    q, k = np.repeat(q, r, 1), np.repeat(k, r, 1)
    lam = np.exp(np.asarray(g, np.float64))[:, None, None]
    N = len(cu) - 1
    h = np.zeros((N, HV, D, D)) if h0 is None else np.array(h0, np.float64)
    dh = np.zeros((N, HV, D, D)) if dht is None else np.array(dht, np.float64)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for n in range(N):
        S, G = h[n], dh[n]
        for t in range(cu[n], cu[n + 1]):
            S *= lam
            S += k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hkv,hv->hk", S, do[t])
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            G += scale * q[t][:, :, None] * do[t][:, None, :]
            dk[t] = np.einsum("hkv,hv->hk", G, v[t])
            dv[t] = np.einsum("hkv,hk->hv", G, k[t])
            G *= lam
    return dict(dq=dq.reshape(T, H, r, D).sum(2), dk=dk.reshape(T, H, r, D).sum(2), dv=dv, dh0=dh)


# Bounds, from what the kernels round.  With A the same sums over absolute values:
#   bf16 outputs: each term has at most one factor rounded to bf16 (8 significant bits: half an
#   ulp is 2^-8 of the value at most) and fp32 sums of at most a few hundred terms per step
#   (2^-12 covers them); the output is rounded once (2^-8).
#   fp32 states: weights good to 2^-21 and fp32 sums whose tensor-core steps may truncate
#   (2^-23 a step, 24 steps a chunk): 2^-18 in all.
def out_bound(ref, mag):
    return (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -7.9 * np.abs(ref) + 1e-30


def state_bound(mag):
    return 2.0 ** -18 * mag + 1e-30


def check(name, got, ref, bound):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, name
    assert np.all(np.isfinite(got)), "%s is not finite" % name
    bad = np.abs(got - ref) > bound
    assert not bad.any(), "%s: %d values off, worst %.3g of the bound" % (
        name, int(bad.sum()), float(np.max(np.abs(got - ref) / bound)))


def rope(x, pos, freq, layout, mscale=1.0, backward=False):
    """Rotation of x [T, h, D] in 64 bits; freq [2, rot / 2] in turns (head + tail)."""
    x = np.asarray(x, np.float64)
    f = np.asarray(freq, np.float64).sum(0)
    p = np.asarray(pos, np.int64).astype(np.float64)
    ang = 2.0 * np.pi * np.remainder(p[:, None] * f, 1.0)[:, None]
    c, s = mscale * np.cos(ang), mscale * np.sin(ang) * (-1.0 if backward else 1.0)
    half = len(f)
    one, two = ((slice(0, half), slice(half, 2 * half)) if layout == "half"
                else (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))
    y = x.copy()
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y
