"""64-bit references of the short convolution, the selective scan and the norms (torch, from their
definitions), with error bounds for the kernels that compute them.

Bounds.  A result in type t is rounded once, by at most half a step (HALF[t] of its value).  What comes
before is fp32: a sum of n products is off by at most (n + 1) 2^-24 of the sum of their absolute values
(`mag` below: the same formula over absolute values), and the sigmoids and softplus, from the hardware's
exponential (2^-22, and 2^-24 |x| by its rounded argument) and reciprocal, by 2^-19 of their values for
|x| <= 16."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(name, got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), "%s is not finite" % name
    bad = (got - ref).abs() > bound
    assert not bad.any(), "%s: %d values off, worst %.3g of the bound" % (
        name, int(bad.sum()), float(((got - ref).abs() / bound).nan_to_num().max()))


def spans(cu):
    return [(n, int(cu[n]), int(cu[n + 1])) for n in range(len(cu) - 1)]


def silu_slope(u):
    s = torch.sigmoid(u)
    return s + u * s * (1 - s)


# ------------------------------------------------------------------------------ convolution
def conv(x, w, cu, bias=None, silu=True, h0=None, dy=None, dht=None):
    """y and the final state; with dy also dx, dw, dbias, dh0.  Each as (value, magnitude)."""
    T, C = x.shape
    W = w.shape[1]
    N = len(cu) - 1
    d = dict(dtype=torch.float64, device=x.device)
    x, w = x.double(), w.double()
    b = torch.zeros(C, **d) if bias is None else bias.double()
    h0 = torch.zeros(N, C, W - 1, **d) if h0 is None else h0.double()
    dht = torch.zeros(N, C, W - 1, **d) if dht is None else dht.double()
    y, ym, ht = torch.zeros(T, C, **d), torch.zeros(T, C, **d), torch.zeros(N, C, W - 1, **d)
    g = {k: torch.zeros(s, **d) for k, s in dict(dx=(T, C), dw=(C, W), db=(C,), dh0=(N, C, W - 1)).items()}
    m = {k: v.clone() for k, v in g.items()}
    for n, a, e in spans(cu):
        rows = torch.cat([h0[n].t(), x[a:e]])
        L = e - a
        ht[n] = rows[L:].t()
        win = torch.stack([rows[j:j + L] for j in range(W)], 2)     # [L, C, W]
        u, um = (win * w).sum(2) + b, (win * w).abs().sum(2) + b.abs()
        act = u * torch.sigmoid(u) if silu else u
        y[a:e] = act
        # u is off by (W + 2) 2^-24 um, which silu passes on by 1.1 at most; the sigmoid by 2^-19
        ym[a:e] = 1.1 * (W + 2) * 2.0 ** -24 * um + 2.0 ** -19 * act.abs()
        if dy is None:
            continue
        do = dy[a:e].double()
        slope = silu_slope(u) if silu else torch.ones_like(u)
        # silu's slope: its two terms by 2^-18 of 1.3 at most, its own slope is at most 0.5
        dd = do * slope
        off = do.abs() * (1.3 * 2.0 ** -18 + 0.5 * (W + 2) * 2.0 ** -24 * um)
        drows, orows = torch.zeros_like(rows), torch.zeros_like(rows)
        drows[L:] += dht[n].t()
        orows[L:] += 2.0 ** -23 * dht[n].t().abs()
        for j in range(W):
            drows[j:j + L] += dd * w[:, j]
            orows[j:j + L] += (off + (W + 2) * 2.0 ** -24 * dd.abs()) * w[:, j].abs()
            g["dw"][:, j] += (dd * win[:, :, j]).sum(0)
            # (sums of a tile's 128 tokens one by one, then of the tiles: fewer than 256 roundings)
            m["dw"][:, j] += ((off + 2.0 ** -16 * dd.abs()) * win[:, :, j].abs()).sum(0)
        g["db"] += dd.sum(0)
        m["db"] += (off + 2.0 ** -16 * dd.abs()).sum(0)
        g["dx"][a:e], m["dx"][a:e] = drows[W - 1:], orows[W - 1:]
        g["dh0"][n], m["dh0"][n] = drows[:W - 1].t(), orows[:W - 1].t()
    return (y, ym), ht, g, m


# ------------------------------------------------------------------------------ scan
def _walk(x, d, A, B, C, D, gate, cu, h0, do, dht, r):
    """The recurrence and its gradient with respect to x, d, A, B, C, D and the states, token by token.
    B, C: [T, C, Ns] already; do: the gradient of the ungated output."""
    T, Ch = x.shape
    y, last = torch.zeros_like(x), h0.clone()
    g = dict(dx=torch.zeros_like(x), dd=torch.zeros_like(x), A=torch.zeros_like(A), B=torch.zeros_like(B),
             C=torch.zeros_like(C), dh0=dht.clone())
    for n, a, e in spans(cu):
        h, seen = h0[n], []
        for t in range(a, e):
            seen.append(h)
            h = torch.exp(d[t, :, None] * A) * h + (d[t] * x[t])[:, None] * B[t]
            y[t] = (C[t] * h).sum(1)
            if do is not None:
                g["C"][t] = do[t][:, None] * h
        last[n] = h
        if do is None:
            continue
        G = dht[n]
        for t in range(e - 1, a - 1, -1):
            G = G + do[t][:, None] * C[t]
            g["B"][t] = G * (d[t] * x[t])[:, None]
            gB = (G * B[t]).sum(1)
            decay = torch.exp(d[t, :, None] * A)
            p = G * decay * seen[t - a]
            g["dd"][t] = (p * (A if r > 0 else A.abs())).sum(1) + gB * x[t]
            g["A"] += p * d[t][:, None]
            g["dx"][t] = gB * d[t]
            G = decay * G
        g["dh0"][n] = G
    return y, last, g


def scan(x, dt, A_log, B, C, cu, D=None, z=None, bias=None, h0=None, dy=None, dht=None):
    """y and the final state; with dy also the gradients.  Each as (value, bound without its rounding)."""
    T, Ch = x.shape
    _, G, Ns = B.shape
    N, r = len(cu) - 1, Ch // G
    f = lambda t, *s: torch.zeros(*s, dtype=torch.float64, device=x.device) if t is None else t.double()  # noqa: E731
    x, Bx, Cx = x.double(), B.double().repeat_interleave(r, 1), C.double().repeat_interleave(r, 1)
    D, bias, h0, dht = f(D, Ch), f(bias, Ch), f(h0, N, Ch, Ns), f(dht, N, Ch, Ns)
    u = dt.double() + bias
    d = torch.nn.functional.softplus(u, threshold=40)
    A = -torch.exp(A_log.double())
    zd = None if z is None else z.double()
    gate = torch.ones_like(x) if z is None else zd * torch.sigmoid(zd)
    do = None if dy is None else dy.double() * gate
    y, last, g = _walk(x, d, A, Bx, Cx, D, gate, cu, h0, do, dht, 1)
    absdo = None if do is None else do.abs()
    ya, lasta, ga = _walk(x.abs(), d, A, Bx.abs(), Cx.abs(), D.abs(), gate.abs(), cu, h0.abs(), absdo, dht.abs(), -1)
    # A state is a sum of inputs times products of decays.  A decay e^{-v} is off by 2^-18 v (d by 2^-19, A and
    # the product by 2^-22) and 2^-22; over a product the first is at most 2^-18 v e^{-v} < 2^-19 of 1, the
    # second n 2^-22 after n tokens, and each token adds two roundings: (n + 4) 2^-21 and 2^-17 cover them.
    n = max([e - a for _, a, e in spans(cu)] + [1])
    rel = 2.0 ** -17 + (n + 4) * 2.0 ** -21
    pre, prea = y + D * x, ya + (D * x).abs()
    out = {"y": (pre * gate, prea * gate.abs() * (rel + 2.0 ** -18)), "ht": (last, lasta * rel)}
    if dy is None:
        return out
    sums = lambda t: t.reshape(T, G, r, Ns).sum(2)  # noqa: E731
    slope = torch.sigmoid(u)
    # a gradient is a product of two such sums (twice the error), summed over states, channels or tokens
    # (at most 2^10 roundings one after another)
    two = 2 * rel + 2.0 ** -14
    du, dua = g["dd"] * slope, ga["dd"] * slope
    out["dx"] = (g["dx"] + D * do, (ga["dx"] + (D * do).abs()) * two)
    out["ddt"] = (du, dua * two)
    out["dA_log"] = (g["A"] * A, ga["A"] * A.abs() * two)
    out["dB"], out["dC"] = ((sums(g[k]), sums(ga[k]) * two) for k in "BC")
    out["dD"] = ((do * x).sum(0), (do * x).abs().sum(0) * two)
    out["ddt_bias"] = (du.sum(0), dua.sum(0) * two)
    out["dh0"] = (g["dh0"], ga["dh0"] * two)
    if z is not None:
        # (the two terms of silu's slope may cancel)
        s = torch.sigmoid(zd)
        out["dz"] = (dy.double() * pre * silu_slope(zd), dy.double().abs() * prea * (s + zd.abs() * s * (1 - s)) * two)
    return out


# ------------------------------------------------------------------------------ norm
def gate_of(kind, z):
    s = torch.sigmoid(z)
    if kind == "sigmoid":
        return s, s * (1 - s), s * (1 - s)
    return z * s, silu_slope(z), s + z.abs() * s * (1 - s)


# 2^-17 of an output: the row's mean (at most 2^-19 of it), 1 / sqrt, the sigmoid (2^-19) and products
REL = 2.0 ** -17


def norm(h, w, z=None, gate="silu", eps=1e-6, offset=0.0):
    """y of rows h, with its magnitude."""
    h, w = h.double(), offset + w.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w
    # (offset + w rounds once, of the larger of the two)
    mag = y.abs() + (y / w).nan_to_num().abs() * abs(offset) * 2.0 ** -6
    if z is not None:
        f = gate_of(gate, z.double())[0]
        y, mag = y * f, mag * f.abs()
    return y, mag * REL


def norm_bwd(h, w, dy, z=None, dh=None, scale=None, x=None, gate="silu", eps=1e-6, offset=0.0):
    """Gradients by their formulas, each with its bound."""
    h, w, dy = h.double(), offset + w.double(), dy.double()
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n, out, u, lost = h * r, {}, dy, w.abs() + abs(offset) * 2.0 ** -6
    rows = h.numel() // h.shape[-1]
    if z is not None:
        f, slope, mag = gate_of(gate, z.double())
        out["dz"] = (dy * n * w * slope, (dy * n).abs() * lost * mag * REL)
        u = dy * f
    e, ea = u * w, u.abs() * lost
    flat = lambda t: t.reshape(-1, t.shape[-1]).sum(0)  # noqa: E731
    # (a block's rows one after another, then the blocks: at most rows / 152 + 152 roundings)
    long = REL + (rows / 152 + 160) * 2.0 ** -24
    out["dweight"] = (flat(u * n), flat((u * n).abs()) * long)
    d = r * (e - n * (e * n).mean(-1, keepdim=True))
    da = r * (ea + n.abs() * (ea * n.abs()).mean(-1, keepdim=True)) * REL
    if dh is not None:
        d, da = d + dh.double(), da + dh.double().abs() * 2.0 ** -23
    out["dresidual"] = (d, da)
    if scale is not None:
        xs = x.double()
        out["dscale"] = (flat(d * xs), flat((da + d.abs() * long) * xs.abs()))
        d, da = d * scale.double(), (da + d.abs() * 2.0 ** -23) * scale.double().abs()
    out["dx"] = (d, da)
    return out
