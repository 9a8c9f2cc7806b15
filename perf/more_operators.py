"""Timed cases of what stands around a recurrence in a layer: the short causal convolution, the
selective state space scan and the norms with their gate and residual.

`conv` and `scan` have a packed forward ("fwd"), its gradient ("bwd"), a prefill over the slots of
a pool ("paged") and a step of one token for each row ("step"); `norm` has "fwd" and "bwd".  `run`
computes them with the library's kernels where `own` is true, else in plain fp32 torch operations;
`exact` gives the fp64 values of the definitions.

    conv:  y[t, c] = act(bias[c] + sum_j w[c, j] x[t - (W - 1) + j, c]),   state = the last W - 1 inputs
    scan:  d = softplus(dt + dt_bias),  h[c, n] = exp(-d[c] e^{A_log[c, n]}) h[c, n] + d[c] B[n] x[c],
           y[c] = (sum_n C[n] h[c, n] + D[c] x[c]) silu(z[c])
    norm:  h = residual + scale x (rounded to the residual's type),
           y = h / sqrt(mean(h^2) + eps) (offset + w) act(z)

x, dt, z, y: [T, channels]; B, C: [T, groups, Ns]; w: fp32 [channels, W]; A_log: fp32 [channels, Ns];
conv states: x's type, [N, channels, W - 1]; scan states: fp32 [N, channels, Ns]; pools alike with slots.
"""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-6

# packed lengths ~ U[1, 8192] up to 32768 tokens: the benchmark's ragged pack
PACK_32K = "6969,5218,4188,2211,2522,336,617,136,1436,6663,2472"


# ------------------------------------------------------------------------------- cases
def _conv(form, lens, C, W=4, act="silu", bias=True, dtype="bf16", slots=0, null=0):
    return {"op": "conv", "form": form, "lens": lens, "C": C, "W": W, "act": act, "bias": bias, "dtype": dtype,
            "slots": slots, "null": null}


def _scan(form, lens, C, Ns=16, G=1, gate=True, skip=True, dtype="bf16", slots=0, null=0):
    return {"op": "scan", "form": form, "lens": lens, "C": C, "Ns": Ns, "G": G, "gate": gate, "skip": skip,
            "dtype": dtype, "slots": slots, "null": null}


def _norm(form, rows, D, gate="none", residual="none", scale=False, offset=0.0, dtype="bf16"):
    return {"op": "norm", "form": form, "rows": rows, "D": D, "gate": gate, "residual": residual, "scale": scale,
            "offset": offset, "dtype": dtype}


def listed():
    return [
        # a serving step: the convolution of q, k and v (16, 16 and 32 heads of 128), a tenth of the rows null
        {"name": "conv_step_256", **_conv("step", "256", 8192, slots=512, null=26)},
        # a training forward of the same channels over a ragged pack
        {"name": "conv_fwd_32k_varlen", **_conv("fwd", PACK_32K, 8192)},
        # its gradient over four equal sequences
        {"name": "conv_bwd_4x4096", **_conv("bwd", "4096,4096,4096,4096", 8192)},
        # a serving step of the scan
        {"name": "scan_step_256", **_scan("step", "256", 4096, slots=512, null=26)},
        # three short prompts (one of them a single token) resumed in pool slots, fp32 activations: latency
        {"name": "scan_prefill_short", **_scan("paged", "1,65,447", 2048, dtype="f32", slots=8)},
        # a training forward of four equal sequences
        {"name": "scan_fwd_4x4096", **_scan("fwd", "4096,4096,4096,4096", 4096)},
        # one long document: few sequences, a long scan
        {"name": "scan_fwd_65536_long", **_scan("fwd", "65536", 2048)},
        # the gradient over a ragged pack
        {"name": "scan_bwd_32k_varlen", **_scan("bwd", PACK_32K, 2048)},
        # the gated norm behind the recurrence: 32 heads of 32768 tokens
        {"name": "norm_gated_32k", **_norm("fwd", 32768 * 32, 128, gate="silu")},
        # its gradient, 16384 tokens
        {"name": "norm_gated_bwd_16k", **_norm("bwd", 16384 * 32, 128, gate="silu")},
        # a serving step's residual and norm, two requests: launch latency
        {"name": "norm_residual_step_2", **_norm("fwd", 2, 4096, residual="bf16")},
        # the training gradient between two blocks: fp32 residual stream, scaled branch
        {"name": "norm_residual_bwd_16k", **_norm("bwd", 16384, 4096, residual="f32", scale=True, offset=1.0)},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    n = min(rng.choice([1, 1, 2, 3, 5, 9]), total)
    cuts = sorted(rng.randrange(0, total + 1) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["conv", "conv", "scan", "scan", "scan", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    wide = 2 if dtype == "f32" else 1
    if op == "norm":
        form = rng.choice(["fwd", "bwd"])
        D = rng.choice([64, 96, 128, 256, 1024, 2048, 4096, 5120, 8192, _log_int(rng, 3, 8192)])
        rows = _log_int(rng, 1, max(2, (1 << 26) // wide // D))
        gate = rng.choice(["none", "silu", "sigmoid"])
        residual = rng.choice(["none", "bf16", "f32"]) if dtype == "bf16" else rng.choice(["none", "f32"])
        return _norm(form, rows, D, gate, residual, residual != "none" and rng.random() < 0.5,
                     rng.choice([0.0, 1.0]), dtype)
    form = rng.choice(["fwd", "bwd", "paged", "step"])
    if op == "conv":
        C = rng.choice([256, 1024, 1280, 2048, 4096, 8192, _log_int(rng, 17, 8192)])
        most = min(32000, (1 << 27) // wide // C)
    else:
        C = rng.choice([64, 96, 768, 1536, 2048, 4096, _log_int(rng, 5, 4096)])
        most = min(32000, (1 << 25) // C)
    extra = {}
    if op == "conv":
        extra = {"W": rng.choice([2, 3, 4, 4]), "act": rng.choice(["silu", "silu", "none"]), "bias": rng.random() < 0.6}
    else:
        G = rng.choice([g for g in (1, 1, 2, 4, 8) if C % g == 0])
        Ns = rng.choice([8, 16, 16, 32])
        most = max(1, most * 16 // max(16, Ns))
        extra = {"Ns": Ns, "G": G, "gate": rng.random() < 0.7, "skip": rng.random() < 0.7}
    make = _conv if op == "conv" else _scan
    if form == "step":
        rows = _log_int(rng, 1, 256)
        return make(form, str(rows), C, dtype=dtype, slots=2 * rows + 2, null=rng.randrange(0, rows // 8 + 1), **extra)
    lens = _lens(rng, _log_int(rng, 1, most))
    slots = lens.count(",") + 2 + rng.randrange(0, 4) if form == "paged" else 0
    return make(form, lens, C, dtype=dtype, slots=slots, **extra)


def _lens_of(case):
    return [int(x) for x in case["lens"].split(",")]


# ------------------------------------------------------------------------------ inputs
def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pool(s, g, case, shape, scale, dtype):
    """A pool's slots: each row or sequence has one of its own, null rows have slot 0."""
    n = len(_lens_of(case)) if case["form"] == "paged" else int(case["lens"])
    idx = torch.randperm(case["slots"] - 1, generator=g, device=DEV)[:n] + 1
    idx[torch.randperm(n, generator=g, device=DEV)[:case["null"]]] = 0
    s["idx"] = idx.to(torch.int32)
    s["pool"] = _randn(g, case["slots"], *shape, scale=scale, dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": dict(case)}
    t = _type(case["dtype"])
    if case["op"] == "norm":
        R, D = case["rows"], case["D"]
        s["weight"] = (1.0 - case["offset"]) + _randn(g, D, scale=0.1)
        s["x"] = _randn(g, R, D, dtype=t)
        if case["gate"] != "none":
            s["z"] = _randn(g, R, D, dtype=t)
        if case["residual"] != "none":
            r = _type(case["residual"])
            s["residual"] = _randn(g, R, D, scale=2.0, dtype=r)
            if case["scale"]:
                s["scale"] = 0.5 + _randn(g, D, scale=0.1)
            if case["form"] == "bwd":   # what the forward left: the residual stream behind the branch
                s["h"] = (s["residual"].float() + (s["scale"] * s["x"].float() if case["scale"] else s["x"].float())).to(r)
                s["dh"] = _randn(g, R, D, dtype=r)
        if case["form"] == "bwd":
            s["dy"] = _randn(g, R, D, dtype=t)
        return s
    lens, C = _lens_of(case), case["C"]
    T, N = sum(lens), len(lens)
    if case["form"] != "step":
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
        s["cu_host"], s["cu"], s["lens"] = cu.numpy(), cu.to(DEV), lens
    if case["op"] == "conv":
        W = case["W"]
        s["x"] = _randn(g, T, C, dtype=t)
        s["w"] = _randn(g, C, W, scale=W ** -0.5)
        s["bias"] = _randn(g, C, scale=0.1) if case["bias"] else None
        if case["slots"]:
            _pool(s, g, case, (C, W - 1), 1.0, t)
        else:
            s["h0"] = _randn(g, N, C, W - 1, dtype=t)
    else:
        Ns, G = case["Ns"], case["G"]
        s["x"], s["dt"] = _randn(g, T, C, dtype=t), _randn(g, T, C, scale=0.5, dtype=t)
        s["B"], s["C"] = _randn(g, T, G, Ns, dtype=t), _randn(g, T, G, Ns, dtype=t)
        s["z"] = _randn(g, T, C, dtype=t) if case["gate"] else None
        s["D"] = 1.0 + _randn(g, C, scale=0.1) if case["skip"] else None
        # the usual start of such a layer: rates 1 .. Ns, steps between 0.001 and 0.1
        rates = torch.log(torch.arange(1, Ns + 1, device=DEV, dtype=torch.float32))
        s["A_log"] = rates + _randn(g, C, Ns, scale=0.1)
        step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(C, generator=g, device=DEV))
        s["dt_bias"] = torch.log(torch.expm1(step))
        if case["slots"]:
            _pool(s, g, case, (C, Ns), 0.3, torch.float32)
        else:
            s["h0"] = _randn(g, N, C, Ns, scale=0.3)
    if case["form"] == "bwd":
        s["dy"] = _randn(g, T, C, dtype=t)
        s["dht"] = _randn(g, *s["h0"].shape, scale=0.3, dtype=s["h0"].dtype)
    return s


# ------------------------------------------------------------------ plain forms: convolution
def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _tokens(s):
    """Sequence of each token, and the sequences' lengths."""
    lens = torch.diff(s["cu"]).long()
    ids = torch.arange(lens.numel(), device=DEV)
    return torch.repeat_interleave(ids, lens, output_size=s["x"].shape[0]), lens


def _conv_rows(s, h0):
    """Every sequence's state rows and tokens one behind the other, fp32; the rows of the tokens, of
    the states, and of the last W - 1 of each sequence."""
    c = s["case"]
    tseq, lens = _tokens(s)
    K = c["W"] - 1
    T, N = tseq.numel(), lens.numel()
    token = torch.arange(T, device=DEV) + (tseq + 1) * K
    first = s["cu"][:-1].long() + torch.arange(N, device=DEV) * K
    state = first[:, None] + torch.arange(K, device=DEV)
    ext = torch.empty(T + N * K, c["C"], device=DEV, dtype=torch.float32)
    ext[token] = s["x"].float()
    ext[state] = h0.float().transpose(1, 2)
    return ext, token, state, state + lens[:, None]


def _conv_pre(s, ext, token):
    W = s["case"]["W"]
    pre = sum(ext[token - (W - 1 - j)] * s["w"][:, j] for j in range(W))
    return pre if s["bias"] is None else pre + s["bias"]


def _conv_act(s, pre):
    return pre * _sigmoid(pre) if s["case"]["act"] == "silu" else pre


def _conv_fwd(s, h0):
    ext, token, state, last = _conv_rows(s, h0)
    t = s["x"].dtype
    return _conv_act(s, _conv_pre(s, ext, token)).to(t), ext[last].transpose(1, 2).to(t).contiguous()


def _conv_bwd(s):
    W, t = s["case"]["W"], s["x"].dtype
    ext, token, state, last = _conv_rows(s, s["h0"])
    dpre = s["dy"].float()
    if s["case"]["act"] == "silu":
        pre = _conv_pre(s, ext, token)
        sig = _sigmoid(pre)
        dpre = dpre * (sig + pre * sig * (1.0 - sig))
    dext = torch.zeros_like(ext)
    dext[last] = s["dht"].float().transpose(1, 2)
    dw = []
    for j in range(W):
        at = token - (W - 1 - j)
        dext[at] += dpre * s["w"][:, j]
        dw.append((dpre * ext[at]).sum(0))
    out = {"dx": dext[token].to(t), "dw": torch.stack(dw, 1), "dh0": dext[state].transpose(1, 2).to(t).contiguous()}
    if s["bias"] is not None:
        out["dbias"] = dpre.sum(0)
    return out


def _conv_step(s):
    idx = s["idx"].long()
    live = (idx > 0)[:, None]
    rows = torch.cat([s["pool"][idx], s["x"][:, :, None]], 2)
    pre = (rows.float() * s["w"]).sum(2)
    y = _conv_act(s, pre if s["bias"] is None else pre + s["bias"])
    s["pool"][idx] = torch.where(live[..., None], rows[:, :, 1:], s["pool"][idx])
    return torch.where(live, y, torch.zeros_like(y)).to(s["x"].dtype), s["pool"]


# ------------------------------------------------------------------------- plain forms: scan
def _chunked(s):
    """Rows of the tokens in chunks of one length (a sequence's last one is filled up), the chunk
    counts and the first chunk of each sequence, the length and the most chunks of a sequence."""
    longest = max(s["lens"])
    L = max(1, int(math.sqrt(longest) / 2))
    tseq, lens = _tokens(s)
    nch = (lens + L - 1) // L
    first = torch.cumsum(nch, 0) - nch
    pos = torch.arange(tseq.numel(), device=DEV) - s["cu"].long()[tseq]
    return first[tseq] * L + pos, nch, first, L, -(-longest // L), sum(-(-n // L) for n in s["lens"])


def _recur(a, b, h0, chunks):
    """All h_t = a_t h_{t-1} + b_t of the packed sequences: a, b [T, ...], h0 [N, ...].  Chunks of all
    sequences at once from zero, then their starts one chunk after another, then both together."""
    row, nch, first, L, most, total = chunks
    shape = a.shape[1:]
    w = torch.ones(total * L, *shape, device=DEV, dtype=torch.float32)
    h = torch.zeros(total * L, *shape, device=DEV, dtype=torch.float32)
    w[row], h[row] = a, b
    w, h = w.view(total, L, *shape), h.view(total, L, *shape)
    for i in range(1, L):
        h[:, i].addcmul_(w[:, i], h[:, i - 1])
        w[:, i].mul_(w[:, i - 1])
    start = torch.empty(total + 1, *shape, device=DEV, dtype=torch.float32)   # (one for those that have ended)
    state = h0.float().clone()
    for k in range(most):
        on = (k < nch).view(-1, *[1] * len(shape))
        at = torch.where(k < nch, first + k, torch.full_like(first, total))
        start[at] = state
        at = torch.clamp(at, max=total - 1)
        state = torch.where(on, w[at, -1] * state + h[at, -1], state)
    h.addcmul_(w, start[:-1, None])
    return h.view(total * L, *shape)[row], state


def _scan_terms(s):
    """d, the decays and the inputs of the recurrence, [T, C(, Ns)] in fp32."""
    C, r = s["x"].shape[1], s["x"].shape[1] // s["B"].shape[1]
    u = s["dt"].float() + s["dt_bias"]
    d = torch.where(u > 20.0, u, torch.log1p(torch.exp(torch.clamp(u, max=20.0))))
    rate = -torch.exp(s["A_log"])
    B, Cm = (s[n].float().repeat_interleave(r, 1) for n in ("B", "C"))
    return u, d, rate, torch.exp(d[..., None] * rate), (d * s["x"].float())[..., None] * B, B, Cm


def _scan_out(s, h, Cm):
    y = (h * Cm).sum(-1)
    return y if s["D"] is None else y + s["D"] * s["x"].float()


def _scan_gated(s, y):
    if s["z"] is None:
        return y.to(s["x"].dtype)
    z = s["z"].float()
    return (y * (z * _sigmoid(z))).to(s["x"].dtype)


def _scan_fwd(s, h0):
    u, d, rate, a, b, B, Cm = _scan_terms(s)
    h, last = _recur(a, b, h0, _chunked(s))
    return _scan_gated(s, _scan_out(s, h, Cm)), last


def _reversed_within(s, x):
    """Each sequence's rows in reverse order."""
    tseq, lens = _tokens(s)
    cu = s["cu"].long()
    return x[cu[tseq] + cu[tseq + 1] - 1 - torch.arange(tseq.numel(), device=DEV)]


def _scan_bwd(s):
    u, d, rate, a, b, B, Cm = _scan_terms(s)
    tseq, lens = _tokens(s)
    chunks = _chunked(s)
    x, t = s["x"].float(), s["x"].dtype
    h, _ = _recur(a, b, s["h0"], chunks)
    dy = s["dy"].float()
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sig = _sigmoid(z)
        out["dz"] = (dy * _scan_out(s, h, Cm) * (sig + z * sig * (1.0 - sig))).to(t)
        dy = dy * (z * sig)
    # g_t = a_{t+1} g_{t+1} + C_t dy_t: the recurrence on reversed rows, with the decay of the row before
    rev = _reversed_within(s, a)
    at_first = torch.zeros(tseq.numel(), device=DEV, dtype=torch.bool)
    at_first[s["cu"].long()[:-1][lens > 0]] = True
    shifted = torch.where(at_first[:, None, None], torch.ones_like(rev), torch.roll(rev, 1, 0))
    g, _ = _recur(shifted, _reversed_within(s, Cm * dy[..., None]), s["dht"], chunks)
    g = _reversed_within(s, g)
    gB = (g * B).sum(-1)
    p = g * (h - b)     # g_t a_t h_{t-1}
    dd = (p * rate).sum(-1) + gB * x
    du = torch.where(u > 20.0, dd, dd * _sigmoid(u))
    dx = gB * d
    if s["D"] is not None:
        dx = dx + s["D"] * dy
        out["dD"] = (dy * x).sum(0)
    G, Ns = s["B"].shape[1:]
    T, C = x.shape
    dh0 = s["dht"].clone()
    some = lens > 0
    head = s["cu"].long()[:-1][some]
    dh0[some] = a[head] * g[head]
    out.update(dx=dx.to(t), ddt=du.to(t), ddt_bias=du.sum(0), dA_log=(p * d[..., None]).sum(0) * rate,
               dB=(g * (d * x)[..., None]).view(T, G, C // G, Ns).sum(2).to(t),
               dC=(h * dy[..., None]).view(T, G, C // G, Ns).sum(2).to(t), dh0=dh0)
    return out


def _scan_step(s):
    idx = s["idx"].long()
    live = (idx > 0)[:, None]
    u, d, rate, a, b, B, Cm = _scan_terms(s)
    h = a * s["pool"][idx] + b
    y = _scan_gated(s, _scan_out(s, h, Cm))
    s["pool"][idx] = torch.where(live[..., None], h, s["pool"][idx])
    return torch.where(live, y, torch.zeros_like(y)), s["pool"]


# ------------------------------------------------------------------------- plain forms: norm
def _norm_gate(c, z):
    """The gate's factor and its slope."""
    sig = _sigmoid(z)
    if c["gate"] == "sigmoid":
        return sig, sig * (1.0 - sig)
    return z * sig, sig + z * sig * (1.0 - sig)


def _norm_fwd(s):
    c = s["case"]
    x, out = s["x"].float(), {}
    if "residual" in s:
        h = s["residual"].float() + (x * s["scale"] if c["scale"] else x)
        out["h"] = h.to(s["residual"].dtype)
        x = out["h"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * (c["offset"] + s["weight"])
    if "z" in s:
        y = y * _norm_gate(c, s["z"].float())[0]
    out["y"] = y.to(s["x"].dtype)
    return out


def _norm_bwd(s):
    c, out = s["case"], {}
    h = (s["h"] if "h" in s else s["x"]).float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    n, w, dy = h * r, c["offset"] + s["weight"], s["dy"].float()
    if "z" in s:
        gate, slope = _norm_gate(c, s["z"].float())
        out["dz"] = (dy * n * w * slope).to(s["x"].dtype)
        dy = dy * gate
    out["dweight"] = (dy * n).sum(0)
    dn = dy * w
    d = r * (dn - n * (dn * n).mean(1, keepdim=True))
    if "dh" in s:
        d = d + s["dh"].float()
        out["dresidual"] = d.to(s["h"].dtype)
        if c["scale"]:
            out["dscale"] = (d * s["x"].float()).sum(0)
            d = d * s["scale"]
    out["dx"] = d.to(s["x"].dtype)
    return out


# ---------------------------------------------------------------------------- one pass
def _into_pool(s, forward):
    idx = s["idx"].long()
    y, last = forward(s, s["pool"][idx])
    s["pool"][idx] = last
    return y, s["pool"]


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _norm_fwd(s) if c["form"] == "fwd" else _norm_bwd(s)
    conv = c["op"] == "conv"
    if c["form"] == "step":
        return _conv_step(s) if conv else _scan_step(s)
    if c["form"] == "bwd":
        return _conv_bwd(s) if conv else _scan_bwd(s)
    forward = _conv_fwd if conv else _scan_fwd
    return _into_pool(s, forward) if c["form"] == "paged" else forward(s, s["h0"])


def _own(s):
    import chunked_gated_delta_06_gb300 as gdn

    c = s["case"]
    if c["op"] == "norm":
        kw = dict(gate=c["gate"], eps=EPS, offset=c["offset"])
        if c["form"] == "fwd":
            y, h = gdn.rms_norm_fwd(s["x"], s["weight"], z=s.get("z"), residual=s.get("residual"), scale=s.get("scale"),
                                    **kw)
            return {"y": y} if h is None else {"y": y, "h": h}
        got = gdn.rms_norm_bwd(s.get("h", s["x"]), s["weight"], s["dy"], z=s.get("z"), dh=s.get("dh"),
                               scale=s.get("scale"), x=s["x"] if c["scale"] else None, **kw)
        return {n: v for n, v in got.items() if v is not None}
    if c["op"] == "conv":
        kw = dict(bias=s["bias"], activation=c["act"])
        if c["form"] == "step":
            return gdn.short_conv_step(s["x"], s["w"], s["pool"], s["idx"], **kw), s["pool"]
        cu = s["cu_host"], s["cu"]
        if c["form"] == "paged":
            return gdn.short_conv_prefill_paged(s["x"], s["w"], *cu, s["pool"], s["idx"], **kw), s["pool"]
        if c["form"] == "fwd":
            return gdn.short_conv_fwd(s["x"], s["w"], *cu, initial_state=s["h0"], **kw)
        got = gdn.short_conv_bwd(s["x"], s["w"], s["dy"], *cu, initial_state=s["h0"], d_final_state=s["dht"], **kw)
    else:
        args = s["x"], s["dt"], s["A_log"], s["B"], s["C"]
        kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        if c["form"] == "step":
            return gdn.selective_scan_step(*args, s["pool"], s["idx"], **kw), s["pool"]
        cu = s["cu_host"], s["cu"]
        if c["form"] == "paged":
            return gdn.selective_scan_prefill_paged(*args, *cu, s["pool"], s["idx"], **kw), s["pool"]
        if c["form"] == "fwd":
            return gdn.selective_scan_fwd(*args, *cu, initial_state=s["h0"], **kw)
        got = gdn.selective_scan_bwd(*args, s["dy"], *cu, initial_state=s["h0"], d_final_state=s["dht"], **kw)
    return {n: v for n, v in got.items() if v is not None}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """Bytes: every input read once, every output written once.  Flops: the definition's own sums
    and products, an exponential counted as one."""
    e = 2 if case["dtype"] == "bf16" else 4
    bwd = case["form"] == "bwd"
    if case["op"] == "norm":
        n = case["rows"] * case["D"]
        gate, scale = case["gate"] != "none", case["scale"]
        r = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
        if bwd:   # h, dy (z, dh, x) in; dx (dz, dresidual) out
            b = (r or e) + 2 * e + 2 * e * gate + 2 * r + e * scale
            return {"bytes": n * b + 4 * case["D"] * (2 + 2 * scale), "flops": 14 * n}
        return {"bytes": n * (2 * e + e * gate + 2 * r) + 4 * case["D"] * (1 + scale), "flops": 6 * n}
    lens, C = _lens_of(case), case["C"]
    T = sum(lens)
    if case["op"] == "conv":
        W = case["W"]
        par = 4 * C * (W + case["bias"])
        if case["form"] == "step":
            live = T - case["null"]
            return {"bytes": e * C * (2 * T + 2 * (W - 1) * live) + par + 4 * T, "flops": 2 * W * C * T}
        state = e * len(lens) * C * (W - 1)
        if bwd:
            return {"bytes": 3 * e * T * C + 3 * state + 2 * par, "flops": (6 * W + 8) * T * C}
        return {"bytes": 2 * e * T * C + 2 * state + par, "flops": (2 * W + 4) * T * C}
    Ns, G, gate = case["Ns"], case["G"], case["gate"]
    par = 4 * C * (Ns + 1 + case["skip"])
    if case["form"] == "step":
        live = T - case["null"]
        return {"bytes": e * T * C * (3 + gate) + 2 * e * T * G * Ns + 8 * live * C * Ns + par + 4 * T,
                "flops": 7 * T * C * Ns}
    state = 4 * len(lens) * C * Ns
    if bwd:
        return {"bytes": e * T * C * (5 + 2 * gate) + 4 * e * T * G * Ns + 3 * state + 2 * par, "flops": 22 * T * C * Ns}
    return {"bytes": e * T * C * (3 + gate) + 2 * e * T * G * Ns + 2 * state + par, "flops": 7 * T * C * Ns}


# ------------------------------------------------------------------------ 64-bit values
def _spans(case):
    at, out = 0, []
    for n in _lens_of(case):
        out.append((at, at + n))
        at += n
    return out


def _exact_conv(s, h0, grads):
    """Windows of each sequence behind its state; gradients by differentiating that."""
    c = s["case"]
    leaf = lambda t: None if t is None else t.double().requires_grad_(grads)  # noqa: E731
    x, w, bias, h0 = leaf(s["x"]), leaf(s["w"]), leaf(s["bias"]), leaf(h0)
    ys, ends = [], []
    for n, (a, b) in enumerate(_spans(c)):
        rows = torch.cat([h0[n].t(), x[a:b]])
        if b > a:
            pre = torch.einsum("tcw,cw->tc", rows.unfold(0, c["W"], 1), w)
            pre = pre if bias is None else pre + bias
            ys.append(torch.nn.functional.silu(pre) if c["act"] == "silu" else pre)
        ends.append(rows[b - a:].t())
    y, last = torch.cat(ys), torch.stack(ends)
    if not grads:
        return y, last
    torch.autograd.backward([y, last], [s["dy"].double(), s["dht"].double()])
    out = {"dx": x.grad, "dw": w.grad, "dh0": h0.grad}
    return out if bias is None else dict(out, dbias=bias.grad)


def _exact_terms(s):
    x, B, Cm = s["x"].double(), s["B"].double(), s["C"].double()
    r = x.shape[1] // B.shape[1]
    u = s["dt"].double() + s["dt_bias"].double()
    d = torch.logaddexp(u, torch.zeros_like(u))
    return x, u, d, -torch.exp(s["A_log"].double()), B, Cm, r


def _exact_scan(s, h0):
    """Token by token."""
    x, u, d, rate, B, Cm, r = _exact_terms(s)
    y, last = torch.empty_like(x), h0.double().clone()
    G, Ns = B.shape[1:]
    for n, (a, b) in enumerate(_spans(s["case"])):
        h = last[n]
        by_group = h.view(G, r, Ns)
        for t in range(a, b):
            h.mul_(torch.exp(d[t, :, None] * rate))
            by_group.add_((d[t] * x[t]).view(G, r, 1) * B[t, :, None])
            y[t] = torch.bmm(by_group, Cm[t, :, :, None]).view(-1)
    y = y if s["D"] is None else y + s["D"].double() * x
    return (y if s["z"] is None else y * torch.nn.functional.silu(s["z"].double())), last


def _exact_scan_bwd(s):
    x, u, d, rate, B, Cm, r = _exact_terms(s)
    T, C = x.shape
    G, Ns = B.shape[1:]
    dy, out = s["dy"].double(), {}
    z = None if s["z"] is None else s["z"].double()
    do = dy if z is None else dy * torch.nn.functional.silu(z)
    ydo = torch.empty_like(x)
    dd, dx, dB, dC = torch.empty_like(x), torch.empty_like(x), torch.empty_like(B), torch.empty_like(Cm)
    drate = torch.zeros_like(rate)
    dh0 = s["dht"].double().clone()
    for n, (a, b) in enumerate(_spans(s["case"])):
        h, before = s["h0"][n].double(), []
        for t in range(a, b):
            before.append(h)
            h = torch.exp(d[t, :, None] * rate) * h + ((d[t] * x[t]).view(G, r, 1) * B[t, :, None]).view(C, Ns)
        g = dh0[n]
        for t in range(b - 1, a - 1, -1):
            g = g + (do[t].view(G, r, 1) * Cm[t, :, None]).view(C, Ns)
            hb = h.view(G, r, Ns)
            ydo[t] = torch.bmm(hb, Cm[t, :, :, None]).view(-1)
            dC[t] = torch.bmm(do[t].view(G, 1, r), hb)[:, 0]
            gb = g.view(G, r, Ns)
            dB[t] = torch.bmm((d[t] * x[t]).view(G, 1, r), gb)[:, 0]
            through = torch.bmm(gb, B[t, :, :, None]).view(-1)
            h = before.pop()
            decay = torch.exp(d[t, :, None] * rate)
            g = g * decay
            gh = g * h
            dd[t] = (gh * rate).sum(1) + through * x[t]
            drate += gh * d[t, :, None]
            dx[t] = through * d[t]
        dh0[n] = g
    if s["D"] is not None:
        D = s["D"].double()
        out["dD"] = (do * x).sum(0)
        dx = dx + D * do
        ydo = ydo + D * x
    if z is not None:
        sig = torch.sigmoid(z)
        out["dz"] = dy * ydo * (sig * (1.0 + z * (1.0 - sig)))
    du = dd * torch.sigmoid(u)
    out.update(dx=dx, ddt=du, ddt_bias=du.sum(0), dA_log=drate * rate, dB=dB, dC=dC, dh0=dh0)
    return out


def _exact_norm(s):
    c = s["case"]
    bwd = c["form"] == "bwd"
    leaf = lambda n: s[n].double().requires_grad_(bwd) if n in s else None  # noqa: E731
    x, w, z, scale = leaf("x"), leaf("weight"), leaf("z"), leaf("scale")
    res, h, out = leaf("residual"), x, {}
    if res is not None:
        h = res + (x if scale is None else x * scale)
        # the norm is of the stream as it is held: its rounding passes gradients through
        held = (s["h"] if bwd else (s["residual"].float() + (s["x"].float() if scale is None else s["scale"] * s["x"].float()))
                .to(s["residual"].dtype)).double()
        out["h"] = h.detach()
        h = h + (held - h).detach()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * (c["offset"] + w)
    if z is not None:
        y = y * (torch.sigmoid(z) if c["gate"] == "sigmoid" else torch.nn.functional.silu(z))
    if not bwd:
        return dict(out, y=y)
    torch.autograd.backward([y] if res is None else [y, h], [s["dy"].double()] + ([] if res is None else [s["dh"].double()]))
    out = {"dx": x.grad, "dweight": w.grad}
    for name, t in (("dz", z), ("dresidual", res), ("dscale", scale)):
        if t is not None:
            out[name] = t.grad
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    conv = case["op"] == "conv"
    if case["form"] == "bwd":
        return _exact_conv(s, s["h0"], True) if conv else _exact_scan_bwd(s)
    forward = (lambda s, h: _exact_conv(s, h, False)) if conv else _exact_scan
    if case["form"] == "fwd":
        return forward(s, s["h0"])
    idx, pool = s["idx"].long(), s["pool"].double()
    if case["form"] == "step":   # every row is a sequence of one token
        s["case"]["lens"] = ",".join(["1"] * len(idx))
    y, last = forward(s, s["pool"][idx])
    live = idx > 0
    pool[idx[live]] = last[live].double()
    return torch.where(live[:, None], y, torch.zeros_like(y)) if case["form"] == "step" else y, pool
