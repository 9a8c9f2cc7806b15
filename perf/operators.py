"""Timed cases of the decay-only linear attention and of the rotary positions.

Four calls are covered: `fwd` (a packed chunk forward, or a paged prefill over the decode
pool's slots), `bwd` (its backward), `step` (one token for each row over the state pool) and
`rope` (rotary positions of q and k, forward or gradient).  `run` computes them with the
library's kernels where `own` is true, else in plain fp32 torch operations; `exact` gives the
fp64 values of the token-by-token definition.

    S_t = e^{g} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   g = log_decay[value head] <= 0

q, k: bf16 [T, H, 128]; v, o: bf16 [T, HV, 128], key head of value head hv = hv // (HV / H);
states fp32 [N, HV, K, V], pool fp32 [slots, HV, V, K].
"""
import math

import torch

own = False
DEV = "cuda"
D = 128
SCALE = D ** -0.5


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a serving step of two requests: launch latency
        {"name": "step_2", "kind": "step", "rows": 2, "H": 16, "HV": 32, "slots": 8, "null": 0},
        # the decode workload of the benchmark: 256 rows, a tenth of them null
        {"name": "step_256", "kind": "step", "rows": 256, "H": 16, "HV": 32, "slots": 512, "null": 26},
        # three short prompts (one of them a single token) resumed in pool slots: latency
        {"name": "prefill_short", "kind": "fwd", "lens": "1,65,447", "H": 8, "HV": 8, "paged": True, "slots": 8},
        # a training forward of four equal sequences
        {"name": "fwd_4x4096", "kind": "fwd", "lens": "4096,4096,4096,4096", "H": 16, "HV": 32, "paged": False,
         "slots": 0},
        # a training forward of a ragged pack
        {"name": "fwd_32k_varlen", "kind": "fwd", "lens": PACK_32K, "H": 16, "HV": 32, "paged": False, "slots": 0},
        # one long document: few sequences, a long scan
        {"name": "fwd_65536_long", "kind": "fwd", "lens": "65536", "H": 16, "HV": 64, "paged": False, "slots": 0},
        # the gradient of a small ragged batch without shared key heads: latency
        {"name": "bwd_short", "kind": "bwd", "lens": "70,1,130", "H": 4, "HV": 4},
        # the training backward of four equal sequences
        {"name": "bwd_4x4096", "kind": "bwd", "lens": "4096,4096,4096,4096", "H": 16, "HV": 32},
        # the training backward of the ragged pack
        {"name": "bwd_32k_varlen", "kind": "bwd", "lens": PACK_32K, "H": 16, "HV": 32},
        # a serving step's positions: half layout, half of each head rotated, far positions
        {"name": "rope_step_256", "kind": "rope", "T": 256, "Hq": 32, "Hk": 8, "D": 128, "rot": 64,
         "layout": "half", "scaling": "none", "backward": False, "max_pos": 131072},
        # a training pack's positions: half layout, whole heads
        {"name": "rope_32k", "kind": "rope", "T": 32768, "Hq": 16, "Hk": 16, "D": 128, "rot": 128,
         "layout": "half", "scaling": "linear", "backward": False, "max_pos": 32768},
        # the gradient of an interleaved layout, part of wider heads, scaled by parts
        {"name": "rope_16k_grad", "kind": "rope", "T": 16384, "Hq": 32, "Hk": 4, "D": 256, "rot": 64,
         "layout": "interleaved", "scaling": "parts", "backward": True, "max_pos": 131072},
    ]


# packed lengths ~ U[1, 8192] up to 32768 tokens: the benchmark's ragged pack
PACK_32K = "6969,5218,4188,2211,2522,336,617,136,1436,6663,2472"


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    n = rng.choice([1, 1, 2, 3, 5, 9])
    n = min(n, total)
    cuts = sorted(rng.randrange(0, total + 1) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def _heads(rng, most):
    H = rng.choice([1, 2, 4, 5, 8, 16])
    r = rng.choice([1, 1, 2, 3, 4])
    while H * r > most:
        r = max(1, r - 1)
        H = H if H * r <= most else H // 2
    return H, H * r


def draw(rng):
    kind = rng.choice(["step", "fwd", "fwd", "bwd", "bwd", "rope"])
    if kind == "step":
        H, HV = _heads(rng, 32)
        rows = _log_int(rng, 1, 256)
        return {"kind": kind, "rows": rows, "H": H, "HV": HV, "slots": 2 * rows + 2,
                "null": rng.randrange(0, rows // 8 + 1)}
    if kind in ("fwd", "bwd"):
        H, HV = _heads(rng, 64 if kind == "fwd" else 32)
        T = _log_int(rng, 1, 60000 if kind == "fwd" else 32000)
        T += T == 3072
        lens = _lens(rng, T)
        case = {"kind": kind, "lens": lens, "H": H, "HV": HV}
        if kind == "fwd":
            n = lens.count(",") + 1
            case["paged"] = rng.random() < 0.5
            case["slots"] = n + 1 + rng.randrange(0, 4) if case["paged"] else 0
        return case
    dim = rng.choice([64, 96, 128, 192, 256])
    T = _log_int(rng, 1, 32768)
    T += T == 3072
    Hq = rng.choice([1, 2, 4, 8, 16])
    return {"kind": kind, "T": T, "Hq": Hq, "Hk": rng.choice([h for h in (1, 2, 4, 8, 16) if h <= Hq]), "D": dim,
            "rot": rng.choice([dim // 4, dim // 2, dim]) if T * Hq * dim <= 1 << 26 else dim // 2,
            "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "parts"]),
            "backward": rng.random() < 0.5, "max_pos": rng.choice([4096, 32768, 131072])}


def _lens_of(case):
    return [int(x) for x in case["lens"].split(",")]


# ------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale


def _bf(x):
    return x.to(torch.bfloat16)


def _decays(HV):
    # geometric slopes from about -0.84 to -1/256, the last head without a decay: a fast and a
    # slow head of such a layer, and plain linear attention
    s = torch.exp2(-8.0 * torch.arange(1, HV + 1, device=DEV, dtype=torch.float64) / HV)
    s[-1] = 0.0
    return (-s).to(torch.float32)


def _frequencies(rot, scaling):
    """float64 rotation of each pair for one position, in turns, for context scaling."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot) / (2.0 * math.pi)
    factor, trained = 4.0, 32768.0
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":  # few turns within the trained length: interpolate; many: keep
        keep = ((f * trained - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f


def _mscale(scaling):
    return 0.1 * math.log(4.0) + 1.0 if scaling == "parts" else 1.0


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    if case["kind"] == "rope":
        T, rot = case["T"], case["rot"]
        s["q"], s["k"] = (_bf(_randn(g, T, case[h], case["D"])) for h in ("Hq", "Hk"))
        s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=g, device=DEV, dtype=torch.int32)
        f = _frequencies(rot, case["scaling"])
        head = f.to(torch.float32)
        s["freq"] = torch.stack([head, (f - head.double()).to(torch.float32)]).to(DEV)  # f as head + tail
        s["mscale"] = _mscale(case["scaling"])
        return s
    H, HV = case["H"], case["HV"]
    s["g"] = _decays(HV)
    if case["kind"] == "step":
        B = case["rows"]
        perm = torch.randperm(case["slots"] - 1, generator=g, device=DEV)[:B] + 1
        perm[torch.randperm(B, generator=g, device=DEV)[:case["null"]]] = 0
        s["idx"] = perm.to(torch.int32)
        T = B
        s["pool"] = _randn(g, case["slots"], HV, D, D, scale=0.1)
    else:
        lens = _lens_of(case)
        T = sum(lens)
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
        s["cu_host"], s["cu"] = cu.numpy(), cu.to(DEV)
        s["lens"] = lens
    # activations as they leave the projections: q and k behind a sigmoid-weighted unit
    s["q"], s["k"] = (_bf(torch.nn.functional.silu(_randn(g, T, H, D))) for _ in range(2))
    s["v"] = _bf(_randn(g, T, HV, D))
    if case["kind"] == "fwd" and case["paged"]:
        s["pool"] = _randn(g, case["slots"], HV, D, D, scale=0.1)
        s["idx"] = (torch.randperm(case["slots"] - 1, generator=g, device=DEV)[:len(s["lens"])] + 1).to(torch.int32)
    elif case["kind"] in ("fwd", "bwd"):
        s["h0"] = _randn(g, len(s["lens"]), HV, D, D, scale=0.1)
    if case["kind"] == "bwd":
        s["do"] = _bf(_randn(g, T, HV, D))
        s["dht"] = _randn(g, len(s["lens"]), HV, D, D, scale=0.1)
    return s


# ------------------------------------------------------------------------- plain forms
CHUNK = 64


def _chunks(s):
    """Chunk tables of the packed sequences: padded row of each token, and for each chunk its
    sequence, its token offset there and its length."""
    lens = torch.diff(s["cu"]).long()
    T, N = s["q"].shape[0], lens.numel()
    nch = (lens + CHUNK - 1) // CHUNK
    total = sum((n + CHUNK - 1) // CHUNK for n in s["lens"])
    first = torch.cumsum(nch, 0) - nch
    ids = torch.arange(N, device=DEV)
    tseq = torch.repeat_interleave(ids, lens, output_size=T)
    row = torch.arange(T, device=DEV) - s["cu"].long()[tseq] + first[tseq] * CHUNK
    cseq = torch.repeat_interleave(ids, nch, output_size=total)
    off = (torch.arange(total, device=DEV) - first[cseq]) * CHUNK
    return row, cseq, off, torch.clamp(lens[cseq] - off, max=CHUNK), lens


def _pad(x, row, n, heads):
    """[T, h, D] -> fp32 [heads, chunk, CHUNK, D], each head repeated for its group."""
    p = torch.zeros(n * CHUNK, x.shape[1], D, device=DEV, dtype=torch.float32)
    p[row] = x.float()
    p = p.permute(1, 0, 2).reshape(x.shape[1], n, CHUNK, D)
    return p.repeat_interleave(heads // x.shape[1], 0)


def _unpad(x, row):
    return x.reshape(x.shape[0], -1, D).permute(1, 0, 2)[row]


def _masked_exp(x, mask):
    return torch.where(mask, torch.exp(torch.where(mask, x, torch.zeros_like(x))), torch.zeros_like(x))


def _plain_states(s, h0):
    """Everything the forward and the backward share."""
    row, cseq, off, L, lens = _chunks(s)
    g = s["g"]
    HV, n = g.numel(), cseq.numel()
    q, k, v = (_pad(s[x], row, n, HV) for x in ("q", "k", "v"))
    i = torch.arange(CHUNK, device=DEV)
    gi = g[:, None, None]
    tril = (i[:, None] >= i[None, :])[None].expand(HV, -1, -1)
    dec = _masked_exp(gi * (i[:, None] - i[None, :]), tril)                     # [HV, C, C]
    into = torch.exp(gi * (i + 1.0)[None, :]).unsqueeze(1).transpose(2, 3)      # [HV, 1, C, 1]
    left = (L[:, None] - 1 - i[None, :])[None].expand(HV, -1, -1)
    w = _masked_exp(gi * left, left >= 0).unsqueeze(3)                          # [HV, n, C, 1]
    kv = (k * w).transpose(2, 3) @ v                                            # [HV, n, K, V]
    same = cseq[:, None] == cseq[None, :]
    gap = (off[:, None] - off[None, :] - CHUNK)
    link = _masked_exp(gi * gap[None], (same & (gap >= 0))[None].expand(HV, -1, -1))
    S = (link @ kv.reshape(HV, n, -1)).reshape(kv.shape)
    S = S + torch.exp(gi * off[None, :, None]).unsqueeze(3) * h0.transpose(0, 1)[:, cseq]
    end = lens[:, None] - off[None, :] - L[None, :]
    mine = torch.arange(lens.numel(), device=DEV)[:, None] == cseq[None, :]
    last = _masked_exp(gi * end[None], mine[None].expand(HV, -1, -1))           # [HV, N, n]
    return row, cseq, off, L, lens, q, k, v, gi, dec, into, w, kv, link, S, last


def _plain_fwd(s, h0):
    row, cseq, off, L, lens, q, k, v, gi, dec, into, w, kv, link, S, last = _plain_states(s, h0)
    A = (q @ k.transpose(2, 3)) * dec[:, None]
    o = SCALE * (A @ v + into * (q @ S))
    fin = (last @ kv.reshape(*kv.shape[:2], -1)).reshape(kv.shape[0], -1, D, D)
    fin = fin.transpose(0, 1) + torch.exp(gi[:, 0] * lens[None, :]).t()[:, :, None, None] * h0
    return _bf(_unpad(o, row)), fin


def _plain_bwd(s):
    h0, dht = s["h0"], s["dht"]
    row, cseq, off, L, lens, q, k, v, gi, dec, into, w, kv, link, S, last = _plain_states(s, h0)
    do = _pad(s["do"], row, cseq.numel(), gi.shape[0])
    HV, n = q.shape[:2]
    A = (q @ k.transpose(2, 3)) * dec[:, None]
    dA = (do @ v.transpose(2, 3)) * dec[:, None]
    gq = SCALE * (q * into).transpose(2, 3) @ do          # each chunk's own part of the state's gradient
    dS = (link.transpose(1, 2) @ gq.reshape(HV, n, -1)).reshape(gq.shape)
    end = (lens[cseq] - off - L).float()
    dS = dS + torch.exp(gi * end[None, :, None]).unsqueeze(3) * dht.transpose(0, 1)[:, cseq]
    dq = SCALE * (dA @ k + into * (do @ S.transpose(2, 3)))
    dk = SCALE * (dA.transpose(2, 3) @ q) + w * (v @ dS.transpose(2, 3))
    dv = SCALE * (A.transpose(2, 3) @ do) + w * (k @ dS)
    mine = torch.arange(lens.numel(), device=DEV)[:, None] == cseq[None, :]
    head = _masked_exp(gi * off[None, None, :].float(), mine[None].expand(HV, -1, -1))
    dh0 = (head @ gq.reshape(HV, n, -1)).reshape(HV, -1, D, D).transpose(0, 1)
    dh0 = dh0 + torch.exp(gi[:, 0] * lens[None, :]).t()[:, :, None, None] * dht
    H = s["q"].shape[1]
    dq, dk = (_unpad(x.reshape(H, HV // H, n, CHUNK, D).sum(1), row) for x in (dq, dk))
    return {"dq": _bf(dq), "dk": _bf(dk), "dv": _bf(_unpad(dv, row)), "dh0": dh0}


def _plain_prefill(s):
    idx = s["idx"].long()
    o, fin = _plain_fwd(s, s["pool"][idx].transpose(2, 3))
    s["pool"][idx] = fin.transpose(2, 3).contiguous()
    return o, s["pool"]


def _plain_step(s):
    idx, r = s["idx"].long(), s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[x].float().repeat_interleave(r, 1) for x in ("q", "k"))
    S = s["pool"][idx] * torch.exp(s["g"])[None, :, None, None] + s["v"].float()[..., None] * k[:, :, None, :]
    o = SCALE * (S * q[:, :, None, :]).sum(3)
    live = (idx > 0)[:, None, None]
    # null rows write nothing: their slot (0, which no live row names) keeps what it holds
    s["pool"][idx] = torch.where(live[..., None], S, s["pool"][idx])
    return _bf(torch.where(live, o, torch.zeros_like(o))), s["pool"]


def _plain_rope(s):
    c = s["case"]
    R = c["rot"]
    pos = s["pos"].float()[:, None]
    turns = pos * s["freq"][0] + pos * s["freq"][1]
    ang = (turns - torch.floor(turns)) * (2.0 * math.pi)
    cos, sin = (torch.cos(ang) * s["mscale"])[:, None], (torch.sin(ang) * s["mscale"])[:, None]
    sin = -sin if c["backward"] else sin
    one, two = ((slice(0, R // 2), slice(R // 2, R)) if c["layout"] == "half"
                else (slice(0, R, 2), slice(1, R, 2)))

    def turn(x):
        x = x.float()
        y = x.clone()
        y[..., one] = x[..., one] * cos - x[..., two] * sin
        y[..., two] = x[..., two] * cos + x[..., one] * sin
        return _bf(y)

    return turn(s["q"]), turn(s["k"])


# ---------------------------------------------------------------------------- one pass
def _own(s):
    import chunked_gated_delta_06_gb300 as gdn

    c = s["case"]
    if c["kind"] == "rope":
        return gdn.rope(s["q"], s["k"], s["pos"], s["freq"], layout=c["layout"], mscale=s["mscale"],
                        backward=c["backward"])
    if c["kind"] == "step":
        return gdn.linear_attn_step(s["q"], s["k"], s["v"], s["g"], s["pool"], s["idx"]), s["pool"]
    if c["kind"] == "bwd":
        return gdn.linear_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["cu_host"], s["cu"],
                                   initial_state=s["h0"], d_final_state=s["dht"])
    if c["paged"]:
        o = gdn.linear_attn_prefill_paged(s["q"], s["k"], s["v"], s["g"], s["cu_host"], s["cu"], s["pool"], s["idx"])
        return o, s["pool"]
    return gdn.linear_attn_fwd(s["q"], s["k"], s["v"], s["g"], s["cu_host"], s["cu"], initial_state=s["h0"])


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "rope":
        return _plain_rope(state)
    if kind == "step":
        return _plain_step(state)
    if kind == "bwd":
        return _plain_bwd(state)
    return _plain_prefill(state) if state["case"]["paged"] else _plain_fwd(state, state["h0"])


def work(case):
    """Bytes: every input read once, every output written once.  Flops: the recurrence's own
    products (one outer product and one matrix-vector product a token and direction)."""
    if case["kind"] == "rope":
        n = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 4 * n * case["D"] + 4 * case["T"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    H, HV = case["H"], case["HV"]
    state = 4 * D * D * HV
    if case["kind"] == "step":
        B, live = case["rows"], case["rows"] - case["null"]
        return {"bytes": 2 * live * state + 2 * B * D * (2 * H + 2 * HV) + 4 * (HV + B), "flops": 4 * D * D * HV * live}
    lens = _lens_of(case)
    T, N = sum(lens), len(lens)
    if case["kind"] == "fwd":
        return {"bytes": 2 * T * D * (2 * H + 2 * HV) + 2 * N * state + 4 * (HV + N + 1), "flops": 4 * D * D * HV * T}
    return {"bytes": 2 * T * D * (4 * H + 3 * HV) + 3 * N * state + 4 * (HV + N + 1), "flops": 10 * D * D * HV * T}


# ------------------------------------------------------------------------ 64-bit values
def _spans(case):
    at, out = 0, []
    for n in _lens_of(case):
        out.append((at, at + n))
        at += n
    return out


def _exact_fwd(s, h0):
    """Token by token from the definition, [HV, K, V] states in fp64."""
    r = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[x].double().repeat_interleave(r, 1) for x in ("q", "k"))
    v, lam = s["v"].double(), torch.exp(s["g"].double())[:, None, None]
    o, fin = torch.empty_like(v), h0.double().clone()
    for n, (a, b) in enumerate(_spans(s["case"])):
        S = fin[n]
        for t in range(a, b):
            S.mul_(lam).addcmul_(k[t].unsqueeze(2), v[t].unsqueeze(1))
            o[t] = torch.bmm(q[t].unsqueeze(1), S).squeeze(1)
    return o * SCALE, fin


def _exact_bwd(s):
    H, HV = s["q"].shape[1], s["v"].shape[1]
    q, k = (s[x].double().repeat_interleave(HV // H, 1) for x in ("q", "k"))
    v, do, lam = s["v"].double(), s["do"].double(), torch.exp(s["g"].double())[:, None, None]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    h, dh = s["h0"].double().clone(), s["dht"].double().clone()
    for n, (a, b) in enumerate(_spans(s["case"])):
        S, G = h[n], dh[n]
        for t in range(a, b):
            S.mul_(lam).addcmul_(k[t].unsqueeze(2), v[t].unsqueeze(1))
            dq[t] = torch.bmm(S, do[t].unsqueeze(2)).squeeze(2)
        for t in range(b - 1, a - 1, -1):
            G.addcmul_(q[t].unsqueeze(2), do[t].unsqueeze(1), value=SCALE)
            dk[t] = torch.bmm(G, v[t].unsqueeze(2)).squeeze(2)
            dv[t] = torch.bmm(k[t].unsqueeze(1), G).squeeze(1)
            G.mul_(lam)
    dq, dk = (x.reshape(x.shape[0], H, -1, D).sum(2) for x in (SCALE * dq, dk))
    return {"dq": dq, "dk": dk, "dv": dv, "dh0": dh}


def _exact_rope(s):
    c = s["case"]
    f = s["freq"].double().sum(0)
    z = torch.polar(torch.full_like(f, s["mscale"])[None].expand(len(s["pos"]), -1),
                    torch.remainder(s["pos"].double()[:, None] * f, 1.0) * (2.0 * math.pi))
    z = (z.conj() if c["backward"] else z)[:, None]
    out = []
    for x in (s["q"].double(), s["k"].double()):
        rot, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        half = c["layout"] == "half"
        pairs = rot.unflatten(-1, (2, -1)).transpose(-1, -2) if half else rot.unflatten(-1, (-1, 2))
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        out.append(torch.cat([(y.transpose(-1, -2) if half else y).flatten(-2), rest], -1))
    return tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_rope(s)
    if case["kind"] == "bwd":
        return _exact_bwd(s)
    if case["kind"] == "fwd":
        if not case["paged"]:
            return _exact_fwd(s, s["h0"])
        idx = s["idx"].long()
        o, fin = _exact_fwd(s, s["pool"][idx].transpose(2, 3))
        pool = s["pool"].double()
        pool[idx] = fin.transpose(2, 3)
        return o, pool
    pool, o = s["pool"].double(), torch.zeros_like(s["v"], dtype=torch.float64)
    r = s["v"].shape[1] // s["q"].shape[1]
    lam = torch.exp(s["g"].double())[:, None, None]
    for b, slot in enumerate(s["idx"].tolist()):
        if slot <= 0:
            continue
        k, q = (s[x][b].double().repeat_interleave(r, 0) for x in ("k", "q"))
        pool[slot] = lam * pool[slot] + torch.einsum("hv,hk->hvk", s["v"][b].double(), k)
        o[b] = SCALE * torch.einsum("hvk,hk->hv", pool[slot], q)
    return o, pool
