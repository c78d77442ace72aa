"""The operators around the LM head, as a measured set of cases.

Each case is one call (or a forward with its backward) of: the residual add + RMS norm in its bf16 and its 8-bit
form and its backward, the 8-bit head product with a power-of-two scale per block of 128, the clipped policy loss with
a KL term, and the preference loss on paired log ratios.  ``run`` computes them in plain 32-bit torch operations, or,
where ``own`` is true, through the library's entry points; ``exact`` states the definitions once more in 64 bits.
"""

import math

import torch

own = False

IGNORE = -100
BLOCK = 128
E4M3_MAX = 448.0
DEV = "cuda"


# ----------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding step's last norm before the 8-bit head: a single token, where latency counts
        {"name": "norm fp8 1x2048", "op": "norm", "T": 1, "Hd": 2048, "x": "bf16", "res": "bf16", "out": "fp8", "pad": 0},
        # a ragged batch of a wide model whose residual stream is kept in 32 bits
        {"name": "norm fp8 1531x4112 f32", "op": "norm", "T": 1531, "Hd": 4112, "x": "bf16", "res": "f32", "out": "fp8", "pad": 0},
        # the norm of the 65,536-token training and scoring workload
        {"name": "norm fp8 65536x2048", "op": "norm", "T": 65536, "Hd": 2048, "x": "bf16", "res": "bf16", "out": "fp8", "pad": 0},
        # the training norm of the policy-gradient batch (8 x 4096), forward and backward with a residual gradient
        {"name": "norm fwd+bwd 32768x2048", "op": "norm_train", "T": 32768, "Hd": 2048, "x": "bf16", "res": "bf16", "dh": True, "pad": 0},
        # logits of one decoding step of one sequence
        {"name": "linear fp8 1x2048x124160", "op": "linear", "T": 1, "K": 2048, "V": 124160},
        # a ragged decoding batch over the whole vocabulary of a two-rank split
        {"name": "linear fp8 93x4096x248320", "op": "linear", "T": 93, "K": 4096, "V": 248320},
        # odd sizes: V not a multiple of anything, a K that ends inside a block of 128
        {"name": "linear fp8 301x1040x4097", "op": "linear", "T": 301, "K": 1040, "V": 4097},
        # a prompt's logits (8192 tokens, the medium workload)
        {"name": "linear fp8 8192x2048x124160", "op": "linear", "T": 8192, "K": 2048, "V": 124160},
        # the policy-gradient batch: 8 sequences of 4096, 30 % prompt, token mean, k3 KL against a reference
        {"name": "policy 8x4096", "op": "policy", "T": 32768, "S": 8, "mask": 0.3, "reduction": "mean", "kl": "k3", "dual": 0.0, "per_seq": False},
        # ragged long rollouts, advantages per sequence, the mean of sequence means, dual clip, garbage in masked places
        {"name": "policy 131072 seqs", "op": "policy", "T": 131072, "S": 61, "mask": 0.2, "reduction": "sequence_mean", "kl": "k2", "dual": 3.0, "per_seq": True},
        # a small preference batch: 16 pairs of short answers
        {"name": "preference 16 pairs", "op": "preference", "P": 16, "mean_len": 200, "mask": 0.4, "kind": "sigmoid", "norm": False, "ref": True},
        # a large one: 128 ragged pairs of long answers, length-normalised
        {"name": "preference 128 long pairs", "op": "preference", "P": 128, "mean_len": 4096, "mask": 0.2, "kind": "ipo", "norm": True, "ref": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "linear", "policy", "preference"])
    if op in ("norm", "norm_train"):
        Hd = 16 * _log_int(rng, 4, 512)
        T = _log_int(rng, 1, min(65536, (1 << 27 if op == "norm" else 1 << 26) // Hd))
        c = {"op": op, "T": T, "Hd": Hd, "x": rng.choice(["bf16", "bf16", "f32"]), "res": rng.choice(["bf16", "f32", "none"]),
             "pad": rng.choice([0, 0, 64])}
        if T * Hd > 1 << 25:
            c["x"] = "bf16"
            c["res"] = "bf16" if c["res"] == "f32" else c["res"]
        if op == "norm":
            c["out"] = rng.choice(["fp8", "bf16", "both"])
        else:
            c["dh"] = rng.random() < 0.5
        return c
    if op == "linear":
        K = 16 * _log_int(rng, 4, 256)
        V = _log_int(rng, 256, 248320)
        T = _log_int(rng, 1, max(1, min(8192, 8192 * 2048 * 124160 // (K * V), 8192 * 124160 // V)))
        return {"op": op, "T": T, "K": K, "V": V}
    if op == "policy":
        T = _log_int(rng, 64, 131072)
        return {"op": op, "T": T, "S": _log_int(rng, 1, max(1, T // 16)), "mask": round(rng.uniform(0.0, 0.9), 3),
                "reduction": rng.choice(["mean", "sequence_mean", "sum"]), "kl": rng.choice(["k1", "k2", "k3"]),
                "dual": rng.choice([0.0, 3.0]), "per_seq": rng.random() < 0.5}
    P = _log_int(rng, 1, 128)
    return {"op": op, "P": P, "mean_len": _log_int(rng, 8, 4096), "mask": round(rng.uniform(0.0, 0.7), 3),
            "kind": rng.choice(["sigmoid", "hinge", "ipo"]), "norm": rng.random() < 0.5, "ref": rng.random() < 0.8}


# ----------------------------------------------------------------------------------------------------- inputs
_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05
BETA, SMOOTH, EPS = 0.1, 0.05, 1e-6


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _lengths(g, n, total_mean):
    """n ragged lengths around total_mean (at least 1)."""
    u = torch.rand(n, generator=g, device=DEV) * 1.5 + 0.25
    return (u * total_mean).long().clamp_(min=1)


def _cu(lengths, T):
    """Offsets of sequences with these relative lengths that fill T tokens (a short one can come out empty)."""
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), lengths.cumsum(0)])
    return cu * T // cu[-1]


def _quantize(y, rows):
    """e4m3 values and E8M0 scales of y [R, K] in blocks of `rows` x 128: the layout the head's weights and the
    normed hidden states come in."""
    R, K = y.shape
    nr, nb = -(-R // rows), -(-K // BLOCK)
    a = torch.zeros(nr * rows, nb * BLOCK, device=y.device)
    a[:R, :K] = y
    amax = a.abs().view(nr, rows, nb, BLOCK).amax(dim=(1, 3))
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1)
    e = (e - 9 + (m > 0.875).int()).clamp(min=-126)
    s = torch.ldexp(torch.ones_like(amax), e)
    q = (a.view(nr, rows, nb, BLOCK) / s[:, None, :, None]).view(nr * rows, nb * BLOCK)[:R, :K]
    return q.contiguous().to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    if c["op"] in ("norm", "norm_train"):
        T, Hd = c["T"], c["Hd"]

        def rows(kind, scale):  # a [T, Hd] view of rows that may be wider than Hd
            t = _randn(g, T, Hd + c["pad"]) * scale
            if kind == "x":
                t[:, ::257] *= 20.0  # outlier channels
            return t

        s = {"c": c, "x": rows("x", 0.5).to(_TYPE[c["x"]])[:, :Hd],
             "w": (1.0 + 0.1 * _randn(g, Hd)).to(torch.bfloat16), "ws": None}
        s["res"] = rows("r", 2.0).to(_TYPE[c["res"]])[:, :Hd] if c["res"] != "none" else None
        if c["op"] == "norm_train":
            s["dy"] = (_randn(g, T, Hd) * 1e-3).to(torch.bfloat16)
            h_type = s["x"].dtype if s["res"] is None else s["res"].dtype
            s["dh"] = (_randn(g, T, Hd) * 1e-3).to(h_type) if c["dh"] else None
        return s
    if c["op"] == "linear":
        x = _randn(g, c["T"], c["K"])
        x[:, ::257] *= 20.0
        xq, xs = _quantize(x, 1)
        Wq, Ws = _quantize(_randn(g, c["V"], c["K"]) * 0.02, BLOCK)
        return {"c": c, "xq": xq, "xs": xs, "Wq": Wq, "Ws": Ws, "ws": torch.empty(1024, dtype=torch.uint8, device=DEV),
                "y": torch.empty(c["T"], c["V"], dtype=torch.bfloat16, device=DEV)}
    if c["op"] == "policy":
        T, S = c["T"], c["S"]
        cu = _cu(_lengths(g, S, 4096), T)
        logp = torch.rand(T, generator=g, device=DEV).clamp_(min=1e-6).log_() * 1.5
        y = torch.randint(0, 124160, (T,), generator=g, device=DEV)
        pos = torch.arange(T, device=DEV)
        seg = torch.searchsorted(cu[1:].contiguous(), pos, right=True).clamp_(max=S - 1)
        start, n = cu[seg], (cu[seg + 1] - cu[seg])
        y[(pos - start).float() < c["mask"] * n.float()] = IGNORE  # the prompt of each sequence
        old = logp + 0.2 * _randn(g, T)
        ref = logp + 0.4 * _randn(g, T)
        masked = y == IGNORE
        logp = torch.where(masked, torch.zeros_like(logp), logp)
        if c["dual"]:  # rollout engines leave what they like in places that are not trained on
            old[masked] = float("nan")
            ref[masked] = float("-inf")
        adv = _randn(g, S if c["per_seq"] else T)
        return {"c": c, "logp": logp, "old": old, "ref": ref, "adv": adv, "y": y, "cu": cu, "ws": None}
    T = 2 * c["P"] * c["mean_len"]
    cu = _cu(_lengths(g, 2 * c["P"], 4096), T)
    lens = cu[1:] - cu[:-1]
    logp = torch.rand(T, generator=g, device=DEV).clamp_(min=1e-6).log_() * 1.5
    ref = logp + 0.1 * _randn(g, T) if c["ref"] else None
    y = torch.randint(0, 124160, (T,), generator=g, device=DEV)
    pos = torch.arange(T, device=DEV)
    seg = torch.searchsorted(cu[1:].contiguous(), pos, right=True)
    y[(pos - cu[seg]).float() < c["mask"] * lens[seg].float()] = IGNORE
    logp = torch.where(y == IGNORE, torch.zeros_like(logp), logp)
    return {"c": c, "logp": logp, "ref": ref, "y": y, "cu": cu, "lmax": int(lens.max()), "ws": None}


# ----------------------------------------------------------------------------------------------------- one pass
def run(state):
    return {"norm": _norm, "norm_train": _norm_train, "linear": _linear, "policy": _policy,
            "preference": _preference}[state["c"]["op"]](state)


def _norm(s):
    c = s["c"]
    if own:
        import lm_head_linear_gb300 as flce
        y, h, _, q, qs = flce.flce_add_rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, normed=c["out"] != "fp8",
                                                fp8=c["out"] != "bf16")
        return {"h": h if s["res"] is not None else None, "y": y, "q": q, "scale": qs}
    h = s["x"].float() if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["res"].dtype).float()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["w"].float()
    out = {"h": h.to(s["res"].dtype) if s["res"] is not None else None, "y": y.to(torch.bfloat16) if c["out"] != "fp8" else None,
           "q": None, "scale": None}
    if c["out"] != "bf16":
        out["q"], e = _quantize(y, 1)
        out["scale"] = e.view(torch.float8_e8m0fnu)
    return out


def _norm_train(s):
    if own:
        import lm_head_linear_gb300 as flce
        y, h, rstd, _, _ = flce.flce_add_rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, save_rstd=True)
        dx, dw, s["ws"] = flce.flce_add_rms_norm_backward(s["dy"], h, s["w"], rstd, dh=s["dh"], workspace=s["ws"])
        return {"h": h if s["res"] is not None else None, "y": y, "rstd": rstd, "dx": dx, "dw": dw}
    h = s["x"].float() if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["res"].dtype).float()
    rstd = torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS)
    w, dy = s["w"].float(), s["dy"].float()
    y = h * rstd * w
    u = dy * w
    dx = rstd * (u - h * (rstd * rstd * (u * h).mean(dim=1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dw = (dy * (h * rstd)).sum(dim=0)
    h_type = s["x"].dtype if s["res"] is None else s["res"].dtype
    return {"h": h.to(h_type) if s["res"] is not None else None, "y": y.to(torch.bfloat16), "rstd": rstd[:, 0],
            "dx": dx.to(h_type), "dw": dw}


def _dequantize(q, e, rows, dtype):
    s = torch.ldexp(torch.ones(e.shape, dtype=dtype, device=e.device), e.int() - 127)
    s = s.repeat_interleave(rows, dim=0)[:q.shape[0]].repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]
    return q.to(dtype) * s


def _linear(s):
    if own:
        import lm_head_linear_gb300 as flce
        return flce.flce_linear_fp8(s["xq"], s["xs"], s["Wq"], s["Ws"], workspace=s["ws"], out={"y": s["y"]})[0]
    x = _dequantize(s["xq"], s["xs"], 1, torch.float32)
    W = _dequantize(s["Wq"], s["Ws"], BLOCK, torch.float32)
    return (x @ W.t()).to(torch.bfloat16)


def _policy(s):
    c = s["c"]
    if own:
        import lm_head_linear_gb300 as flce
        loss, dlogp, stats, n_valid, s["ws"] = flce.flce_policy_loss(
            s["logp"], s["old"], s["adv"], s["y"], ref_logp=s["ref"], cu_seqlens=s["cu"], per_sequence=c["per_seq"],
            ignore_index=IGNORE, reduction=c["reduction"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, dual_clip=c["dual"],
            kl_coef=KL_COEF, kl=c["kl"], workspace=s["ws"])
        return {"loss": loss, "dlogp": dlogp, "stats": stats, "n_valid": n_valid}
    zero = torch.zeros_like(s["logp"])
    valid = s["y"] != IGNORE
    f = valid.float()
    T, S = c["T"], c["S"]
    seg = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(T, device=DEV), right=True).clamp(max=S - 1)
    A = torch.where(valid, s["adv"][seg] if c["per_seq"] else s["adv"], zero)
    raw = torch.where(valid, s["logp"] - s["old"], zero)
    d = raw.clamp(-20.0, 20.0)
    rho = d.exp()
    up = (A > 0) & (d > math.log1p(CLIP_HIGH))
    down = (A < 0) & (d < math.log1p(-CLIP_LOW))
    dual = (A < 0) & (d > math.log(c["dual"])) if c["dual"] else torch.zeros_like(valid)
    ratio = torch.where(up, 1.0 + CLIP_HIGH, torch.where(down, 1.0 - CLIP_LOW, torch.where(dual, c["dual"], rho)))
    cut = up | down | dual
    e = torch.where(valid, s["ref"] - s["logp"], zero)
    if c["kl"] == "k1":
        kl, dkl = -e, torch.ones_like(e)
    elif c["kl"] == "k2":
        kl, dkl = 0.5 * e * e, -e
    else:
        ec = e.clamp(-20.0, 20.0)
        kl, dkl = torch.expm1(ec) - ec, torch.where(e.abs() > 20.0, zero, -torch.expm1(ec))
    per = torch.where(valid, -A * ratio + KL_COEF * kl, zero)
    grad = torch.where(cut | (raw.abs() > 20.0), zero, -A * rho) + KL_COEF * dkl
    n = valid.sum()
    if c["reduction"] == "mean":
        wt = f / n.clamp(min=1).float()
    elif c["reduction"] == "sum":
        wt = f
    else:
        ns = torch.zeros(S, device=DEV).index_add_(0, seg, f)
        wt = f / (ns[seg].clamp(min=1.0) * (ns > 0).sum().clamp(min=1).float())
    inv = 1.0 / n.clamp(min=1).float()
    stats = torch.stack([(kl * f).sum(), (cut & valid).sum().float(), (d * f).sum(), (rho * f).sum()]) * inv
    return {"loss": (per * wt).sum().reshape(1), "dlogp": grad * wt, "stats": stats, "n_valid": n.reshape(1)}


def _preference(s):
    c = s["c"]
    if own:
        import lm_head_linear_gb300 as flce
        loss, dlogp, chosen, rejected, s["ws"] = flce.flce_preference_loss(
            s["logp"], s["y"], s["cu"], ref_logp=s["ref"], ignore_index=IGNORE, reduction="mean", kind=c["kind"], beta=BETA,
            label_smoothing=SMOOTH if c["kind"] == "sigmoid" else 0.0, length_normalize=c["norm"], workspace=s["ws"])
        return {"loss": loss, "dlogp": dlogp, "chosen": chosen, "rejected": rejected}
    valid = s["y"] != IGNORE
    x = torch.where(valid, s["logp"] - s["ref"] if s["ref"] is not None else s["logp"], torch.zeros_like(s["logp"]))
    T = x.shape[0]
    at = s["cu"][:-1, None] + torch.arange(s["lmax"], device=DEV)
    inside = at < s["cu"][1:, None]
    at = at.clamp(max=T - 1)
    S = torch.where(inside, x[at], torch.zeros((), device=DEV)).sum(dim=1)
    n = (inside & valid[at]).sum(dim=1).clamp(min=1).float()
    if c["norm"]:
        S = S / n
    D = S[0::2] - S[1::2]
    h = BETA * D
    if c["kind"] == "sigmoid":
        per = (1 - SMOOTH) * _softplus(-h) + SMOOTH * _softplus(h)
        g = BETA * (SMOOTH * _sigmoid(h) - (1 - SMOOTH) * _sigmoid(-h))
    elif c["kind"] == "hinge":
        per, g = (1.0 - h).clamp(min=0.0), torch.where(h < 1.0, -BETA, 0.0)
    else:
        m = D - 1.0 / (2.0 * BETA)
        per, g = m * m, 2.0 * m
    g = g / c["P"]
    gs = torch.stack([g, -g], dim=1).reshape(-1)
    if c["norm"]:
        gs = gs / n
    seg = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(T, device=DEV), right=True)
    return {"loss": per.mean().reshape(1), "dlogp": torch.where(valid, gs[seg], torch.zeros_like(x)),
            "chosen": BETA * S[0::2], "rejected": BETA * S[1::2]}


def _softplus(v):
    return v.clamp(min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


# ----------------------------------------------------------------------------------------------------- work and 64 bits
def work(case):
    c = case
    if c["op"] in ("norm", "norm_train"):
        n = c["T"] * c["Hd"]
        bx = 2 if c["x"] == "bf16" else 4
        br = {"bf16": 2, "f32": 4, "none": 0}[c["res"]]
        b = n * (bx + 2 * br) + 2 * c["Hd"]  # x, residual in and out, the weight
        if c["op"] == "norm":
            b += (n + c["T"] * -(-c["Hd"] // BLOCK) if c["out"] != "bf16" else 0) + (2 * n if c["out"] != "fp8" else 0)
            return {"bytes": b, "flops": 8 * n}
        bh = br or bx
        # y and rstd out; then dy, h, rstd and the upstream gradient in, dx and dw out
        b += 2 * n + 4 * c["T"] + (2 + bh + (bh if c["dh"] else 0) + bh) * n + 4 * c["T"] + 6 * c["Hd"]
        return {"bytes": b, "flops": 18 * n}
    if c["op"] == "linear":
        T, K, V = c["T"], c["K"], c["V"]
        nb = -(-K // BLOCK)
        return {"bytes": T * K + V * K + T * nb + -(-V // BLOCK) * nb + 2 * T * V, "flops": 2 * T * K * V}
    if c["op"] == "policy":
        return {"bytes": c["T"] * (3 * 4 + 8 + 4) + 4 * (c["S"] if c["per_seq"] else c["T"]) + 8 * (c["S"] + 1), "flops": 20 * c["T"]}
    T = 2 * c["P"] * c["mean_len"]
    return {"bytes": T * (4 + (4 if c["ref"] else 0) + 8 + 4) + 16 * c["P"], "flops": 4 * T}


def _e8m0(amax):
    """The exponent of the smallest power of two that brings amax to 448 or less, at least 2^-126."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / E4M3_MAX))
    e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= amax, e - 1, e)
    e = torch.where(torch.exp2(e) * E4M3_MAX < amax, e + 1, e)
    return e.clamp(min=-126)


def _round_e4m3(v):
    """|v| <= 448 to the nearest e4m3 number, ties to even, from the format's definition: 4 significant bits down to
    2^-6, steps of 2^-9 below."""
    p = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(p - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] in ("norm", "norm_train"):
        w = s["w"].double()
        h = s["x"].double()
        if s["res"] is not None:
            h = (h + s["res"].double()).to(s["res"].dtype).double()
        inv = 1.0 / torch.sqrt((h * h).sum(1) / c["Hd"] + EPS)
        xhat = h * inv[:, None]
        y = xhat * w
        if c["op"] == "norm":
            out = {"h": h if s["res"] is not None else None, "y": y if c["out"] != "fp8" else None, "q": None, "scale": None}
            if c["out"] != "bf16":
                nb = -(-c["Hd"] // BLOCK)
                full = torch.nn.functional.pad(y, (0, nb * BLOCK - c["Hd"])).view(c["T"], nb, BLOCK)
                sc = torch.exp2(_e8m0(full.abs().amax(2)))
                out["q"] = _round_e4m3(full / sc[:, :, None]).view(c["T"], -1)[:, :c["Hd"]]
                out["scale"] = sc
            return out
        dy = s["dy"].double()
        u = dy * w
        dx = inv[:, None] * (u - xhat * ((u * xhat).sum(1, keepdim=True) / c["Hd"]))
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"h": h if s["res"] is not None else None, "y": y, "rstd": inv, "dx": dx, "dw": (dy * xhat).sum(0)}
    if c["op"] == "linear":
        return _dequantize(s["xq"], s["xs"], 1, torch.float64) @ _dequantize(s["Wq"], s["Ws"], BLOCK, torch.float64).t()
    if c["op"] == "policy":
        at = (s["y"] != IGNORE).nonzero()[:, 0]  # only the trained tokens
        seg = (torch.searchsorted(s["cu"], at, right=True) - 1).clamp(max=c["S"] - 1)
        lp = s["logp"].double()[at]
        A = (s["adv"].double()[seg] if c["per_seq"] else s["adv"].double()[at])
        x = lp - s["old"].double()[at]
        d = x.clamp(-20, 20)
        r = torch.exp(d)
        hi, lo = 1 + CLIP_HIGH, 1 - CLIP_LOW
        obj = torch.minimum(r * A, r.clamp(lo, hi) * A)
        live = torch.where(A > 0, r <= hi, torch.where(A < 0, r >= lo, True))
        if c["dual"]:
            capped = (A < 0) & (r > c["dual"])
            obj = torch.where(capped, c["dual"] * A, obj)
            live = live & ~capped
        k = lp - s["ref"].double()[at]
        if c["kl"] == "k1":
            kl, dk = k, torch.ones_like(k)
        elif c["kl"] == "k2":
            kl, dk = k * k / 2, k
        else:
            kc = k.clamp(-20, 20)
            kl, dk = torch.expm1(-kc) + kc, torch.where(k.abs() > 20, 0.0, -torch.expm1(-kc))
        n = at.numel()
        if c["reduction"] == "mean":
            wt = torch.full_like(lp, 1.0 / max(n, 1))
        elif c["reduction"] == "sum":
            wt = torch.ones_like(lp)
        else:
            ns = torch.bincount(seg, minlength=c["S"]).double()
            wt = 1.0 / (ns[seg] * max(int((ns > 0).sum()), 1))
        dl = torch.zeros(c["T"], dtype=torch.float64, device=DEV)
        dl[at] = wt * (torch.where(live & (x.abs() <= 20), -A * r, 0.0) + KL_COEF * dk)
        stats = torch.stack([kl.sum(), (~live).double().sum(), d.sum(), r.sum()]) / max(n, 1)
        return {"loss": (wt * (KL_COEF * kl - obj)).sum().reshape(1), "dlogp": dl, "stats": stats, "n_valid": None}
    v = s["y"] != IGNORE
    x = s["logp"].double() - (s["ref"].double() if s["ref"] is not None else 0.0)
    x = torch.where(v, x, 0.0)
    seg = torch.searchsorted(s["cu"], torch.arange(x.numel(), device=DEV), right=True) - 1
    tot = torch.zeros(2 * c["P"], dtype=torch.float64, device=DEV).index_add_(0, seg, x)
    cnt = torch.bincount(seg[v], minlength=2 * c["P"]).double().clamp(min=1)
    if c["norm"]:
        tot = tot / cnt
    D = (tot[0::2] - tot[1::2]).requires_grad_(True)
    if c["kind"] == "sigmoid":
        sp = torch.nn.functional.softplus
        per = (1 - SMOOTH) * sp(-BETA * D, threshold=1e9) + SMOOTH * sp(BETA * D, threshold=1e9)
    elif c["kind"] == "hinge":
        per = torch.relu(1 - BETA * D)
    else:
        per = (D - 0.5 / BETA) ** 2
    loss = per.mean()
    (g,) = torch.autograd.grad(loss, D)
    gs = torch.stack([g, -g], 1).reshape(-1)
    if c["norm"]:
        gs = gs / cnt
    return {"loss": loss.detach().reshape(1), "dlogp": torch.where(v, gs[seg], 0.0), "chosen": BETA * tot[0::2],
            "rejected": BETA * tot[1::2]}
