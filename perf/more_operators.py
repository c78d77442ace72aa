"""Operators of a rollout and of its training step around the LM head, as a measured set of cases.

Each case is one call (or a forward with its backward) of: the head's product with 4-bit weights and a power-of-two
scale per group of 32, drawing tokens from logits (temperature, top-k, top-p, min-p) with given random numbers, and the
residual add + RMS norm that keeps its input for the backward in 8 bits.  ``run`` computes them in plain torch
operations, or, where ``own`` is true, through the library's entry points; ``exact`` states the definitions once more
in 64 bits.
"""

import math

import torch

own = False

IGNORE = -100
GROUP = 32   # weights of one 4-bit scale
BLOCK = 128  # channels of one 8-bit scale
E4M3_MAX, E2M1_MAX = 448.0, 6.0
EPS = 1e-6
DEV = "cuda"


# ----------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # logits of one decoding step of one sequence
        {"name": "linear fp4 1x2048x124160", "op": "linear", "T": 1, "K": 2048, "V": 124160},
        # a small decoding batch of a wide model over a vocabulary split in two, an odd number of tokens
        {"name": "linear fp4 17x4096x124160", "op": "linear", "T": 17, "K": 4096, "V": 124160},
        # a ragged decoding batch over the whole vocabulary
        {"name": "linear fp4 93x4096x248320", "op": "linear", "T": 93, "K": 4096, "V": 248320},
        # odd sizes: V not a multiple of anything, a K that ends inside a group
        {"name": "linear fp4 301x1040x4097", "op": "linear", "T": 301, "K": 1040, "V": 4097},
        # a prompt's logits
        {"name": "linear fp4 2048x2048x124160", "op": "linear", "T": 2048, "K": 2048, "V": 124160},
        # one sequence with the usual filters, where latency counts
        {"name": "sample 1x248320", "op": "sample", "T": 1, "V": 248320, "x": "bf16", "mode": "filters", "mask": 0.0, "pad": 0},
        # a batch of rollouts as training wants them: the model's own distribution, 32-bit logits
        {"name": "sample 256x124160 f32 plain", "op": "sample", "T": 256, "V": 124160, "x": "f32", "mode": "plain", "mask": 0.0, "pad": 0},
        # a ragged decoding batch, top-p alone over the whole vocabulary
        {"name": "sample 93x248320 top-p", "op": "sample", "T": 93, "V": 248320, "x": "bf16", "mode": "top_p", "mask": 0.0, "pad": 0},
        # many requests, each with settings of its own (greedy ones among them), logits that a grammar masks, odd vocabulary
        {"name": "sample 777x32001 per row", "op": "sample", "T": 777, "V": 32001, "x": "bf16", "mode": "rows", "mask": 0.3, "pad": 0},
        # the training norm of one long sequence, forward and backward from the 8-bit checkpoint
        {"name": "norm checkpoint 500x2048", "op": "norm", "T": 500, "Hd": 2048, "x": "bf16", "res": "bf16", "dh": True, "pad": 0},
        # a ragged batch of a wide model whose residual stream is kept in 32 bits
        {"name": "norm checkpoint 1531x4112 f32", "op": "norm", "T": 1531, "Hd": 4112, "x": "bf16", "res": "f32", "dh": True, "pad": 0},
        # the training norm of the policy-gradient batch (8 x 4096)
        {"name": "norm checkpoint 32768x2048", "op": "norm", "T": 32768, "Hd": 2048, "x": "bf16", "res": "bf16", "dh": True, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "sample", "norm"])
    if op == "linear":
        K = 16 * _log_int(rng, 4, 256)
        V = _log_int(rng, 256, 248320)
        T = _log_int(rng, 1, max(1, min(2048, 2048 * 2048 * 124160 // (K * V), 2048 * 124160 // V)))
        return {"op": op, "T": T, "K": K, "V": V}
    if op == "sample":
        V = _log_int(rng, 1000, 248320)
        return {"op": op, "T": _log_int(rng, 1, max(1, min(1024, (1 << 24) // V))), "V": V, "x": rng.choice(["bf16", "f32"]),
                "mode": rng.choice(["filters", "plain", "top_p", "top_k", "min_p", "rows"]),
                "mask": rng.choice([0.0, 0.0, round(rng.uniform(0.0, 0.95), 3)]), "pad": rng.choice([0, 0, 1, 64])}
    Hd = 16 * _log_int(rng, 4, 512)
    T = _log_int(rng, 1, min(32768, (1 << 26) // Hd))
    return {"op": op, "T": T, "Hd": Hd, "x": rng.choice(["bf16", "bf16", "f32"]), "res": rng.choice(["bf16", "f32", "none"]),
            "dh": rng.random() < 0.5, "pad": rng.choice([0, 0, 64])}


# ----------------------------------------------------------------------------------------------------- inputs
_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _pow2(e):
    return torch.ldexp(torch.ones(e.shape, device=e.device), e)


def _exponent(amax, top):
    """The exponent of the smallest power of two that brings amax = m 2^e, m in [1/2, 1), to ``top`` or less."""
    m, e = torch.frexp(amax)
    mt, et = math.frexp(top)
    return (e - et + (m > mt).int()).clamp(min=-126)


def _e4m3(y):
    """e4m3 values and scale exponents of y [R, K], one scale per row and 128 channels."""
    R, K = y.shape
    nb = -(-K // BLOCK)
    a = torch.nn.functional.pad(y, (0, nb * BLOCK - K)).view(R, nb, BLOCK)
    e = _exponent(a.abs().amax(dim=2), E4M3_MAX)
    q = (a / _pow2(e)[:, :, None]).view(R, nb * BLOCK)[:, :K]
    return q.contiguous().to(torch.float8_e4m3fn), e


def _e2m1(y):
    """Packed 4-bit codes [R, 64 nb] and scale bytes [nb, R, 4] of y [R, K], nb = ceil(K / 128): the layout the
    head's weights come in (the first of two channels in the low bits, rows padded with zeros to whole blocks)."""
    R, K = y.shape
    nb = -(-K // BLOCK)
    a = torch.nn.functional.pad(y, (0, nb * BLOCK - K)).view(R, 4 * nb, GROUP)
    e = _exponent(a.abs().amax(dim=2), E2M1_MAX).clamp(max=125)
    a = a / _pow2(e)[:, :, None]
    m = a.abs()
    step = torch.where(m < 2.0, 0.5, torch.where(m < 4.0, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=E2M1_MAX)
    code = torch.where(m < 2.0, 2.0 * m, torch.where(m < 4.0, m + 2.0, 0.5 * m + 4.0)).to(torch.uint8)
    code = (code + torch.signbit(a).to(torch.uint8) * 8).view(R, nb * BLOCK // 2, 2)
    return code[:, :, 0] + code[:, :, 1] * 16, (e + 127).to(torch.uint8).view(R, nb, 4).transpose(0, 1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    if c["op"] == "linear":
        x = _randn(g, c["T"], c["K"])
        x[:, ::257] *= 20.0  # outlier channels
        xq, e = _e4m3(x)
        parts = [_e2m1(_randn(g, min(32768, c["V"] - v), c["K"]) * 0.02) for v in range(0, c["V"], 32768)]
        return {"c": c, "xq": xq, "xs": (e + 127).to(torch.uint8), "Wq": torch.cat([p[0] for p in parts]),
                "Ws": torch.cat([p[1] for p in parts], dim=1).contiguous(), "ws": torch.empty(1024, dtype=torch.uint8, device=DEV),
                "y": torch.empty(c["T"], c["V"], dtype=torch.bfloat16, device=DEV)}
    if c["op"] == "sample":
        T, V = c["T"], c["V"]
        # from rows that a few words share to rows where thousands do
        logits = _randn(g, T, V + c["pad"]) * (1.0 + 2.0 * _rand(g, T, 1))
        at = torch.randint(0, V, (T, 24), generator=g, device=DEV)
        logits.scatter_add_(1, at, 14.0 * _rand(g, T, 24))
        if c["mask"]:
            logits[_rand(g, T, V + c["pad"]) < c["mask"]] = float("-inf")
            if T >= 8:
                logits[5] = float("-inf")  # a place of the batch that no request holds
        s = {"c": c, "logits": logits.to(_TYPE[c["x"]])[:, :V], "u": _rand(g, T), "temperature": 1.0, "top_k": 0, "top_p": 1.0,
             "min_p": 0.0}
        mode = c["mode"]
        if mode == "filters":
            s.update(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
        elif mode in ("top_p", "top_k", "min_p"):
            s[mode] = {"top_p": 0.95, "top_k": 200, "min_p": 0.05}[mode]
        elif mode == "rows":
            off = _rand(g, 4, T) < 0.25  # each setting is off for some requests
            s["temperature"] = torch.where(off[0], 0.0, 0.3 + 1.2 * _rand(g, T))
            s["top_k"] = torch.where(off[1], 0, torch.randint(1, 1000, (T,), generator=g, device=DEV)).int()
            s["top_p"] = torch.where(off[2], 1.0, 0.5 + 0.5 * _rand(g, T))
            s["min_p"] = torch.where(off[3], 0.0, 0.1 * _rand(g, T))
        return s
    T, Hd = c["T"], c["Hd"]

    def rows(scale):  # [T, Hd], in rows that may be longer
        t = _randn(g, T, Hd + c["pad"]) * scale
        t[:, ::257] *= 20.0
        return t[:, :Hd]

    h_type = _TYPE[c["x"] if c["res"] == "none" else c["res"]]
    return {"c": c, "x": rows(0.5).to(_TYPE[c["x"]]), "res": rows(2.0).to(h_type) if c["res"] != "none" else None,
            "w": (1.0 + 0.1 * _randn(g, Hd)).to(torch.bfloat16), "dy": (_randn(g, T, Hd) * 1e-3).to(torch.bfloat16),
            "dh": (_randn(g, T, Hd) * 1e-3).to(h_type) if c["dh"] else None, "ws": None}


# ----------------------------------------------------------------------------------------------------- one pass
def run(state):
    return {"linear": _linear, "sample": _sample, "norm": _norm}[state["c"]["op"]](state)


def _dequantize_fp4(q, e, K, dtype):
    """[R, K] values of packed codes and scale bytes [nb, R, 4]."""
    e = e.transpose(0, 1).reshape(q.shape[0], -1)
    code = torch.stack([q & 15, q >> 4], dim=2).view(q.shape[0], -1)
    m = (code & 7).to(dtype)
    m = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    m = torch.where(code >= 8, -m, m).view(q.shape[0], -1, GROUP)
    s = torch.ldexp(torch.ones(e.shape, dtype=dtype, device=e.device), e.int() - 127)
    return (m * s[:, :, None]).view(q.shape[0], -1)[:, :K]


def _dequantize_fp8(q, e, dtype):
    s = torch.ldexp(torch.ones(e.shape, dtype=dtype, device=e.device), e.int())
    return q.to(dtype) * s.repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _linear(s):
    if own:
        import lm_head_linear_gb300 as flce
        return flce.flce_linear_fp4(s["xq"], s["xs"], s["Wq"], s["Ws"], workspace=s["ws"], out={"y": s["y"]})[0]
    x = _dequantize_fp8(s["xq"], s["xs"].int() - 127, torch.float32)
    y = torch.empty(s["c"]["T"], s["c"]["V"], dtype=torch.bfloat16, device=DEV)
    for v in range(0, s["c"]["V"], 32768):
        W = _dequantize_fp4(s["Wq"][v:v + 32768], s["Ws"][:, v:v + 32768], s["c"]["K"], torch.float32)
        y[:, v:v + 32768] = x @ W.t()
    return y


def _sample(s):
    if own:
        import lm_head_linear_gb300 as flce
        tokens, logp = flce.flce_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                        min_p=s["min_p"], ignore_index=IGNORE)
        return {"tokens": tokens, "logp": logp}
    T, V = s["c"]["T"], s["c"]["V"]

    def per_row(v):
        return v.double()[:, None] if torch.is_tensor(v) else torch.full((T, 1), float(v), dtype=torch.float64, device=DEV)

    temp, k, p, mp = per_row(s["temperature"]), per_row(s["top_k"]), per_row(s["top_p"]), per_row(s["min_p"])
    greedy = temp == 0
    top, at = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    best = top[:, :1].double()
    w = torch.exp((top.double() - best) / torch.where(greedy, 1.0, temp))  # sums of up to 248,320 of them: 64 bits
    w = torch.where(torch.isneginf(top), 0.0, w)
    pos = torch.arange(V, device=DEV)[None]
    keep = (k <= 0) | (pos < k)
    keep = torch.where(greedy, pos == 0, keep)
    w = torch.where(keep, w, 0.0)
    before = w.cumsum(dim=1)
    total = before[:, -1:].clone()
    before -= w
    keep = (p >= 1) | (before < p * total) | (pos == 0)
    w = torch.where(keep & (w >= mp), w, 0.0)
    cum = torch.zeros_like(w).scatter_(1, at, w).cumsum(dim=1)
    mass = cum[:, -1:].clone()
    token = torch.searchsorted(cum, s["u"].double()[:, None] * mass, right=True)
    empty = mass[:, 0] == 0
    token = torch.where(empty[:, None], 0, token)
    l = s["logits"].gather(1, token).double()
    logp = torch.where(greedy, 0.0, (l - best) / torch.where(greedy, 1.0, temp) - mass.log())[:, 0]
    return {"tokens": torch.where(empty, IGNORE, token[:, 0]), "logp": torch.where(empty, 0.0, logp).float()}


def _norm(s):
    if own:
        import lm_head_linear_gb300 as flce
        y, h, rstd, q, qs = flce.flce_add_rms_norm_checkpoint(s["x"], s["w"], residual=s["res"], eps=EPS)
        dx, dw, s["ws"] = flce.flce_add_rms_norm_checkpoint_backward(s["dy"], q, qs, s["w"], rstd, dh=s["dh"], dtype=h.dtype,
                                                                     workspace=s["ws"])
        return {"h": h if s["res"] is not None else None, "y": y, "rstd": rstd, "q": q, "scale": qs, "dx": dx, "dw": dw}
    h_type = s["x"].dtype if s["res"] is None else s["res"].dtype
    h = s["x"].float() if s["res"] is None else (s["x"].float() + s["res"].float()).to(h_type).float()
    rstd = torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS)
    w, dy = s["w"].float(), s["dy"].float()
    y = h * rstd * w
    q, e = _e4m3(h)
    kept = _dequantize_fp8(q, e, torch.float32)
    u = dy * w
    dx = rstd * (u - kept * (rstd * rstd * (u * kept).mean(dim=1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dw = (dy * (kept * rstd)).sum(dim=0)
    return {"h": h.to(h_type) if s["res"] is not None else None, "y": y.to(torch.bfloat16), "rstd": rstd[:, 0], "q": q,
            "scale": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu), "dx": dx.to(h_type), "dw": dw}


# ----------------------------------------------------------------------------------------------------- work and 64 bits
def work(case):
    c = case
    if c["op"] == "linear":
        T, K, V = c["T"], c["K"], c["V"]
        return {"bytes": T * K + T * -(-K // BLOCK) + V * K // 2 + V * -(-K // GROUP) + 2 * T * V, "flops": 2 * T * K * V}
    if c["op"] == "sample":
        n = c["T"] * c["V"]
        return {"bytes": n * (2 if c["x"] == "bf16" else 4) + c["T"] * (4 + 12 + (16 if c["mode"] == "rows" else 0)), "flops": 4 * n}
    n, T = c["T"] * c["Hd"], c["T"]
    bx = 2 if c["x"] == "bf16" else 4
    bh = {"bf16": 2, "f32": 4, "none": bx}[c["res"]]
    saved = n + T * -(-c["Hd"] // BLOCK) + 4 * T  # the 8-bit checkpoint and rstd
    b = n * bx + (2 * bh * n if c["res"] != "none" else 0) + 2 * c["Hd"] + 2 * n + saved
    b += 2 * n + saved + (bh * n if c["dh"] else 0) + bh * n + 6 * c["Hd"]
    return {"bytes": b, "flops": 20 * n}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "linear":
        e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        e2m1 = torch.cat([e2m1, -e2m1])
        nb = -(-c["K"] // BLOCK)
        sx = torch.exp2(s["xs"].double() - 127).unsqueeze(2).expand(-1, -1, BLOCK).reshape(c["T"], nb * BLOCK)[:, :c["K"]]
        x = s["xq"].double() * sx
        y = torch.empty(c["T"], c["V"], dtype=torch.float64, device=DEV)
        for v in range(0, c["V"], 16384):
            q = s["Wq"][v:v + 16384].int()
            sw = torch.exp2(s["Ws"][:, v:v + 16384].double() - 127).permute(1, 0, 2).reshape(q.shape[0], 4 * nb)
            W = torch.empty(q.shape[0], nb * BLOCK, dtype=torch.float64, device=DEV)
            W[:, 0::2], W[:, 1::2] = e2m1[q % 16], e2m1[q // 16]
            W *= sw.unsqueeze(2).expand(-1, -1, GROUP).reshape(W.shape)
            y[:, v:v + 16384] = x @ W[:, :c["K"]].t()
        return y
    if c["op"] == "sample":
        tokens, logps = [], []
        setting = {n: (s[n].tolist() if torch.is_tensor(s[n]) else [s[n]] * c["T"]) for n in ("temperature", "top_k", "top_p", "min_p")}
        u = s["u"].tolist()
        for r in range(c["T"]):
            l = s["logits"][r].double()
            ids = (l > -math.inf).nonzero()[:, 0]
            if ids.numel() == 0:
                tokens.append(IGNORE), logps.append(0.0)
                continue
            temp, k, p, mp = (setting[n][r] for n in ("temperature", "top_k", "top_p", "min_p"))
            if temp == 0:
                tokens.append(int((l == l.max()).nonzero()[0, 0])), logps.append(0.0)
                continue
            ids = ids[torch.argsort(-l[ids], stable=True)]  # best first, equal ones by their index
            if 0 < k < ids.numel():
                ids = ids[:k]
            z = (l[ids] - l[ids[0]]) / temp
            q = torch.softmax(z, 0)
            n = ids.numel()
            if p < 1:
                n = min(n, int((q.cumsum(0) < p).sum()) + 1)  # the first prefix that reaches p
            if mp > 0:
                n = min(n, int((q >= mp * q[0]).sum()))
            ids, z = torch.sort(ids[:n])[0], None
            q = torch.softmax(l[ids] / temp, 0)
            i = min(int((q.cumsum(0) <= u[r]).sum()), n - 1)
            tokens.append(int(ids[i])), logps.append(float(torch.log_softmax(l[ids] / temp, 0)[i]))
        return {"tokens": torch.tensor(tokens, device=DEV), "logp": torch.tensor(logps, dtype=torch.float64, device=DEV)}
    w, dy, h = s["w"].double(), s["dy"].double(), s["x"].double()
    if s["res"] is not None:
        h = (h + s["res"].double()).to(s["res"].dtype).double()
    T, Hd = h.shape
    inv = 1.0 / torch.sqrt((h * h).sum(1) / Hd + EPS)
    nb = -(-Hd // BLOCK)
    full = torch.nn.functional.pad(h, (0, nb * BLOCK - Hd)).view(T, nb, BLOCK)
    amax = full.abs().amax(2)
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / E4M3_MAX))
    e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= amax, e - 1, e)
    e = torch.where(torch.exp2(e) * E4M3_MAX < amax, e + 1, e).clamp(min=-126)
    scale = torch.exp2(e)
    v = full / scale[:, :, None]
    # to four significant bits down to 2^-6, in steps of 2^-9 below
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0) - 3)
    q = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    xhat = (q * scale[:, :, None]).view(T, -1)[:, :Hd] * inv[:, None]
    g = dy * w
    dx = inv[:, None] * (g - xhat * ((g * xhat).sum(1, keepdim=True) / Hd))
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"h": h if s["res"] is not None else None, "y": h * inv[:, None] * w, "rstd": inv, "q": q.view(T, -1)[:, :Hd],
            "scale": scale, "dx": dx, "dw": (dy * xhat).sum(0)}
