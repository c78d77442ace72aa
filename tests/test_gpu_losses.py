"""Policy and preference losses against 64-bit formulas, their gradients against
autograd of the formula and against differences, and their refusals.

Bounds.  A log ratio is one fp32 subtraction (at most 2^-24 * 20 off where it is
not exact), exp and expm1 add 2 ulp: every term and gradient is within 2e-6 of
the sum of its parts' magnitudes.  Sums over tokens are fp32 over at most a
few tokens, then 64 bits.
"""

import math

import pytest
import torch

import lm_head_linear_gb300 as flce

pytestmark = pytest.mark.gpu

IGN = -100
TOL = 2e-6


def cu_of(lengths, dev, start=0):
    return torch.tensor([start] + list(torch.tensor(lengths).cumsum(0) + start), dtype=torch.int64, device=dev)


def draw(T, dev, seed=0, mask=0.3, spread=0.3):
    g = torch.Generator(device=dev).manual_seed(seed)
    logp = -torch.rand(T, generator=g, device=dev) * 6
    old = logp + spread * torch.randn(T, generator=g, device=dev)
    ref = logp + 0.5 * torch.randn(T, generator=g, device=dev)
    y = torch.randint(0, 1000, (T,), generator=g, device=dev)
    y[torch.rand(T, generator=g, device=dev) < mask] = IGN
    adv = torch.randn(T, generator=g, device=dev)
    return logp, old, ref, adv, y, g


# --------------------------------------------------------------------------------------------- policy
def policy_reference(logp, old, ref, adv, y, cu=None, per_sequence=False, reduction="mean", clip_low=0.2, clip_high=0.2,
                     dual_clip=0.0, kl_coef=0.0, kl="k3", dloss=None):
    """(loss, dlogp, stats, n, magnitude of each token's gradient, magnitude of the loss) in 64 bits."""
    T = logp.shape[0]
    pos = torch.arange(T, device=logp.device)
    valid = y != IGN
    seg = torch.zeros(T, dtype=torch.int64, device=logp.device)
    S = 1
    if cu is not None:
        S = cu.numel() - 1
        seg = torch.searchsorted(cu, pos, right=True) - 1
        valid = valid & (seg >= 0) & (seg < S)
        seg = seg.clamp(0, max(S - 1, 0))
    lp = logp.double().clone().requires_grad_(True)
    at = valid.nonzero()[:, 0]
    x = lp[at]
    A = (adv.double()[seg[at]] if per_sequence else adv.double()[at])
    d = (x - old.double()[at]).clamp(-20, 20)
    rho = d.exp()
    obj = torch.minimum(rho * A, rho.clamp(1 - clip_low, 1 + clip_high) * A)
    cut = ((A > 0) & (rho > 1 + clip_high)) | ((A < 0) & (rho < 1 - clip_low))
    if dual_clip:
        cut = cut | ((A < 0) & (rho > dual_clip))
        obj = torch.where(A < 0, torch.maximum(obj, dual_clip * A), obj)
    k = torch.zeros_like(x)
    if ref is not None:
        e = ref.double()[at] - x
        k = {"k1": -e, "k2": e * e / 2, "k3": torch.expm1(e.clamp(-20, 20)) - e.clamp(-20, 20)}[kl]
    per = -obj + kl_coef * k
    n = at.numel()
    if reduction == "mean":
        w = torch.full_like(per, 1.0 / max(n, 1))
    elif reduction == "sequence_mean":
        ns = torch.bincount(seg[at], minlength=S).double()
        w = 1.0 / (ns[seg[at]] * max(int((ns > 0).sum()), 1))
    else:
        w = torch.ones_like(per)
    if reduction == "none":
        loss = torch.zeros(T, dtype=torch.float64, device=logp.device).index_put((at,), per)
        up = torch.ones_like(loss) if dloss is None else dloss.double()
        w = w * up[at]
    else:
        loss = (per * w).sum()
        up = torch.ones_like(loss) if dloss is None else dloss.double()[0]
        w = w * up
    (g,) = torch.autograd.grad(loss, lp, up) if n else (torch.zeros_like(lp),)
    mag = torch.zeros(T, dtype=torch.float64, device=logp.device)
    mag[at] = (w.abs() * (A.abs() * rho + abs(kl_coef) * (1 + k.abs() + rho))).detach()
    stats = torch.stack([k.sum(), cut.double().sum(), d.sum(), rho.sum()]).detach() / max(n, 1)
    size = (w.abs() * (obj.abs() + abs(kl_coef) * (k.abs() + 1))).sum().detach()
    return loss.detach(), g, stats, n, mag, size


def check_policy(args, ref_kw, **kw):
    logp, old, ref, adv, y = args
    loss, dlogp, stats, n_valid, ws = flce.flce_policy_loss(logp, old, adv, y, ref_logp=ref, **kw)
    assert flce.flce_read_device_status(ws) == 0
    want, g, st, n, mag, size = policy_reference(logp, old, ref, adv, y, **ref_kw)
    assert int(n_valid) == n
    assert bool(((dlogp.double() - g).abs() <= TOL * mag).all())
    if kw.get("reduction") == "none":
        assert bool(((loss.double() - want).abs() <= TOL * (want.abs() + adv.abs().max() + 1)).all())
        assert bool((loss[y == IGN] == 0).all())
    else:
        assert abs(float(loss) - float(want)) <= TOL * float(size) + 1e-12
    assert bool(((stats.double() - st).abs() <= TOL * (st.abs() + 1)).all())
    assert bool((dlogp[y == IGN] == 0).all())
    return loss, dlogp, stats, ws


@pytest.mark.parametrize("T", [1, 2, 31, 33, 1000, 1025, 4096, 16385, 32768, 32769, 70001, 300007, 1100003])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none", "sequence_mean"])
def test_policy(cuda_device, T, reduction):
    logp, old, ref, adv, y, g = draw(T, cuda_device, seed=T)
    cuts = torch.randint(0, T + 1, (min(T, 40),), generator=g, device=cuda_device).sort().values  # some empty
    cu = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)])
    kl = {0: "k1", 1: "k2", 2: "k3"}[T % 3]
    kw = dict(reduction=reduction, clip_low=0.2, clip_high=0.28, kl_coef=0.05, kl=kl, dual_clip=3.0 if T % 2 else 0.0)
    dloss = torch.randn(T if reduction == "none" else 1, generator=g, device=cuda_device)
    _, dlogp, _, ws = check_policy((logp, old, ref, adv, y), dict(kw, cu=cu, dloss=dloss), cu_seqlens=cu, dloss=dloss, **kw)
    again = flce.flce_policy_loss(logp, old, adv, y, ref_logp=ref, cu_seqlens=cu, dloss=dloss, workspace=ws, **kw)
    assert torch.equal(again[1], dlogp)
    advs = torch.randn(cu.numel() - 1, generator=g, device=cuda_device)
    check_policy((logp, old, ref, advs, y), dict(kw, cu=cu, per_sequence=True), cu_seqlens=cu, per_sequence=True, **kw)
    if reduction != "sequence_mean":
        plain = dict(reduction=reduction)
        check_policy((logp, old, None, adv, y), plain, **plain)


@pytest.mark.parametrize("reduction", ["mean", "sequence_mean", "sum", "none"])
def test_policy_masks(cuda_device, reduction):
    """Nothing valid, one valid token, sequences without a valid token, tokens in no sequence, an empty
    batch; NaN and infinities in masked places reach nothing."""
    T = 3000
    logp, old, ref, adv, y, _ = draw(T, cuda_device, seed=5)
    cu = cu_of([0, 700, 0, 0, 900, 1100, 0], cuda_device, start=150)  # 150 before, 150 after
    kw = dict(reduction=reduction, kl_coef=0.1, kl="k3")
    for keep in ([], [800], [149, 150], [2849, 2850, 2999], range(900, 1000), range(T)):
        yy = torch.full_like(y, IGN)
        for t in keep:
            yy[t] = 3
        loss, dlogp, stats, _ = check_policy((logp, old, ref, adv, yy), dict(kw, cu=cu), cu_seqlens=cu, **kw)
        if not any(150 <= t < 2850 for t in keep):
            assert bool((dlogp == 0).all()) and bool((loss == 0).all()) and bool((stats == 0).all())
        bad = [t.clone() for t in (logp, old, ref, adv)]
        for v, t in zip((float("nan"), float("-inf"), float("inf"), float("nan")), bad):
            t[yy == IGN] = v
            t[:150] = v
            t[2850:] = v
        loss2, dlogp2, stats2, _, _ = flce.flce_policy_loss(bad[0], bad[1], bad[3], yy, ref_logp=bad[2], cu_seqlens=cu, **kw)
        assert torch.equal(dlogp, dlogp2) and torch.equal(loss, loss2) and torch.equal(stats, stats2)
    e = torch.empty(0, device=cuda_device)
    ye = torch.empty(0, dtype=torch.int64, device=cuda_device)
    cu0 = torch.zeros(1, dtype=torch.int64, device=cuda_device)
    loss, dlogp, stats, n, _ = flce.flce_policy_loss(e, e, e, ye, cu_seqlens=cu0, reduction=reduction)
    assert dlogp.numel() == 0 and int(n) == 0 and bool((stats == 0).all()) and bool((loss == 0).all())


@pytest.mark.parametrize("T,S", [(5000, 4500), (32768, 4095), (32768, 9000), (60000, 4095), (60000, 4096), (200000, 30000)])
@pytest.mark.parametrize("reduction", ["sequence_mean", "mean"])
def test_policy_many_sequences(cuda_device, T, S, reduction):
    """More offsets than shared memory keeps, with empty and fully masked sequences among them."""
    logp, old, ref, adv, y, g = draw(T, cuda_device, seed=S, mask=0.5)
    cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device=cuda_device).sort().values
    cu = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)])
    advs = torch.randn(S, generator=g, device=cuda_device)
    kw = dict(reduction=reduction, kl_coef=0.05, kl="k3")
    check_policy((logp, old, ref, advs, y), dict(kw, cu=cu, per_sequence=True), cu_seqlens=cu, per_sequence=True, **kw)


@pytest.mark.parametrize("T", [100, 50000])
def test_policy_without_sequences(cuda_device, T):
    """No sequence at all: no token counts."""
    logp, old, _, adv, y, _ = draw(T, cuda_device)
    cu = torch.zeros(1, dtype=torch.int64, device=cuda_device)
    for red in ("mean", "sequence_mean", "sum", "none"):
        loss, dlogp, stats, n, ws = flce.flce_policy_loss(logp, old, adv, y, cu_seqlens=cu, reduction=red)
        assert bool((loss == 0).all()) and bool((dlogp == 0).all()) and bool((stats == 0).all()) and int(n) == 0
        assert flce.flce_read_device_status(ws) == 0


def test_policy_extreme_ratios(cuda_device):
    """Log ratios far beyond the clamp stay finite and carry no gradient from the ratio; a NaN in a trained
    token is not hidden; zero advantages and exact clip borders."""
    d = torch.tensor([0.0, 25.0, -25.0, 90.0, -90.0, 20.0, -20.0, 5.0, -5.0, 0.1, math.inf, -math.inf], device=cuda_device)
    for A in (1.0, -1.0, 0.0):
        n = d.numel()
        logp = torch.full((n,), -3.0, device=cuda_device)
        logp[-2], logp[-1] = 0.0, 0.0
        old = logp - d
        adv = torch.full((n,), A, device=cuda_device)
        y = torch.zeros(n, dtype=torch.int64, device=cuda_device)
        loss, dlogp, _, _, _ = flce.flce_policy_loss(logp, old, adv, y, reduction="none")
        dc = d.double().clamp(-20, 20)
        rho = dc.exp()
        want = -torch.minimum(rho * A, rho.clamp(0.8, 1.2) * A)
        assert bool(((loss.double() - want).abs() <= TOL * want.abs()).all())
        live = (d.abs() <= 20) & ((rho <= 1.2) if A > 0 else (rho >= 0.8) if A < 0 else torch.ones_like(d, dtype=torch.bool))
        want_g = torch.where(live, -A * rho, 0.0)
        assert bool(((dlogp.double() - want_g).abs() <= TOL * want_g.abs()).all())
        old[3] = float("nan")
        loss, dlogp, _, _, _ = flce.flce_policy_loss(logp, old, adv, y, reduction="none")
        assert bool(torch.isnan(loss[3])) and int(torch.isnan(loss).sum()) == 1


def test_policy_autograd_and_differences(cuda_device):
    logp, old, ref, adv, y, g = draw(400, cuda_device, seed=9, spread=0.15)
    cu = cu_of([100, 0, 250, 50], cuda_device)
    kw = dict(reduction="sequence_mean", kl_coef=0.2, kl="k3", clip_low=0.2, clip_high=0.3)
    x = logp.clone().requires_grad_(True)
    loss, stats = flce.policy_loss(x, old, adv, y, ref, cu, **kw)
    (2.5 * loss).backward()
    assert not stats.requires_grad
    # keep away from the kinks: differences are taken on tokens that are not near a clip border
    d = (logp - old).double()
    smooth = ((d - math.log(1.3)).abs() > 1e-3) & ((d - math.log(0.8)).abs() > 1e-3)
    v = torch.randn(400, generator=g, device=cuda_device).double() * smooth
    step = 1e-5
    value = lambda lp: float(policy_reference(lp, old, ref, adv, y, cu=cu, **kw)[0])
    want = 2.5 * (value(logp.double() + step * v) - value(logp.double() - step * v)) / (2 * step)
    assert abs(float((x.grad.double() * v).sum()) - want) <= 1e-5 * float((x.grad.double() * v).abs().sum())
    xn = logp.clone().requires_grad_(True)
    per, _ = flce.policy_loss(xn, old, adv, y, ref, cu, **dict(kw, reduction="none"))
    per.sum().backward()  # an expanded gradient
    want = flce.flce_policy_loss(logp, old, adv, y, ref_logp=ref, cu_seqlens=cu, **dict(kw, reduction="none"))[1]
    assert torch.equal(xn.grad, want)


def test_policy_bad_sequences_are_flagged(cuda_device):
    logp, old, ref, adv, y, _ = draw(1000, cuda_device)
    for cu in ([0, 500, 400, 1000], [0, 500, 1001], [-1, 1000], [2 ** 40, 3]):
        cu = torch.tensor(cu, dtype=torch.int64, device=cuda_device)
        *_, ws = flce.flce_policy_loss(logp, old, adv, y, cu_seqlens=cu, reduction="sequence_mean")
        assert flce.flce_read_device_status(ws) == 8
    big = draw(40000, cuda_device)
    for cu in ([0, 30000, 20000, 40000], [0, 20000, 40001], [-1, 40000], [2 ** 40, 3], [0] * 5000 + [39999, 1, 40000]):
        cu = torch.tensor(cu, dtype=torch.int64, device=cuda_device)
        *_, ws = flce.flce_policy_loss(big[0], big[1], big[3], big[4], cu_seqlens=cu, reduction="sequence_mean")
        assert flce.flce_read_device_status(ws) == 8
    *_, ws = flce.flce_policy_loss(logp, old, adv, y, workspace=ws)
    assert flce.flce_read_device_status(ws) == 0


def test_policy_refusals(cuda_device):
    logp, old, ref, adv, y, _ = draw(16, cuda_device)
    cu = cu_of([16], cuda_device)
    f = flce.flce_policy_loss
    for bad in (dict(clip_low=1.0), dict(clip_low=-0.1), dict(clip_high=-1.0), dict(dual_clip=0.5), dict(kl_coef=0.1),
                dict(reduction="sequence_mean"), dict(kl_coef=float("nan"), ref_logp=ref), dict(forward=False, grad=False)):
        with pytest.raises(flce.FlceError) as e:
            f(logp, old, adv, y, **bad)
        assert e.value.status == 1, bad
    for args, kw in (((logp.cpu(), old, adv, y), {}), ((logp, old[:8], adv, y), {}), ((logp, old, adv.double(), y), {}),
                     ((logp, old, adv, y.int()), {}), ((logp, old, adv, y), dict(cu_seqlens=cu, per_sequence=True)),
                     ((logp, old, adv, y), dict(cu_seqlens=cu.int())), ((logp, old, adv, y), dict(dloss=logp)),
                     ((logp[::2], old[:8], adv[:8], y[:8]), {})):
        with pytest.raises(ValueError):
            f(*args, **kw)
    with pytest.raises(flce.FlceError) as e:
        f(logp, old, adv, y, workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device))
    assert e.value.status == 4


# --------------------------------------------------------------------------------------------- preference
def preference_reference(logp, ref, y, cu, kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0,
                         length_normalize=False, reduction="mean", dloss=None):
    """(loss, dlogp, chosen, rejected, sum of |terms| of each sequence) in 64 bits."""
    T, P = logp.shape[0], cu.numel() // 2
    lp = logp.double().clone().requires_grad_(True)
    valid = y != IGN
    seg = torch.searchsorted(cu, torch.arange(T, device=logp.device), right=True) - 1
    at = (valid & (seg >= 0) & (seg < 2 * P)).nonzero()[:, 0]
    x = lp[at] - (ref.double()[at] if ref is not None else 0.0)
    zero = torch.zeros(2 * P, dtype=torch.float64, device=logp.device)
    n = torch.bincount(seg[at], minlength=2 * P).double().clamp(min=1)
    n = n if length_normalize else torch.ones_like(n)
    S = zero.index_add(0, seg[at], x) / n
    mag = zero.index_add(0, seg[at], x.detach().abs()) / n
    D = S[0::2] - S[1::2]
    h = beta * D - margin
    sp = lambda v: torch.logaddexp(v, torch.zeros_like(v))
    per = {"sigmoid": (1 - label_smoothing) * sp(-h) + label_smoothing * sp(h), "hinge": (1 - h).clamp(min=0),
           "ipo": (D - 1 / (2 * beta)) ** 2}[kind]
    loss = {"mean": per.mean(), "sum": per.sum(), "none": per}[reduction]
    up = torch.ones_like(loss) if dloss is None else dloss.double().reshape(loss.shape)
    (g,) = torch.autograd.grad(loss, lp, up) if at.numel() else (torch.zeros_like(lp),)
    return loss.detach(), g, beta * S[0::2].detach(), beta * S[1::2].detach(), mag, D.detach()


def check_preference(logp, ref, y, cu, dloss=None, longest=1, **kw):
    loss, dlogp, chosen, rejected, ws = flce.flce_preference_loss(logp, y, cu, ref_logp=ref, dloss=dloss, **kw)
    assert flce.flce_read_device_status(ws) == 0
    want, g, c, r, mag, D = preference_reference(logp, ref, y, cu, dloss=dloss, **kw)
    # a sequence's sum: one rounding per term and fp32 chains of longest / 256 + 1 terms
    err = mag * 6e-8 * (3 + longest / 256)
    beta = kw.get("beta", 0.1)
    assert bool(((chosen.double() - c).abs() <= beta * err[0::2] + 2e-7 * c.abs()).all())
    assert bool(((rejected.double() - r).abs() <= beta * err[1::2] + 2e-7 * r.abs()).all())
    dD = err[0::2] + err[1::2] + 1e-7 * D.abs()     # error of D
    h = (beta * D).abs() + abs(kw.get("margin", 0.0)) + 1
    kind = kw.get("kind", "sigmoid")
    if kind == "ipo":
        e_loss = 2 * ((D - 0.5 / beta).abs() + dD) * (dD + 1e-7 * (D.abs() + 0.5 / beta))
        e_slope = 2 * (dD + 1e-7 * (D.abs() + 0.5 / beta))
    else:
        e_loss = beta * dD + 5e-7 * h
        e_slope = beta * (beta * dD + 5e-7 * h)
    red = kw.get("reduction", "mean")
    if red == "none":
        assert bool(((loss.double() - want).abs() <= e_loss + 1e-7 * want.abs()).all())
    else:
        assert abs(float(loss) - float(want)) <= float(e_loss.sum() if red == "sum" else e_loss.mean()) + 2e-7 * abs(float(want))
    if kind == "hinge":  # the slope jumps at h = 1: pairs too near it say nothing
        near = (beta * D - kw.get("margin", 0.0) - 1).abs() <= e_loss
        assert not bool(near.any())
    up = 1.0 if dloss is None else dloss.double().abs().max().item()
    seg = (torch.searchsorted(cu, torch.arange(logp.numel(), device=logp.device), right=True) - 1).clamp(0, 2 * D.numel() - 1)
    assert bool(((dlogp.double() - g).abs() <= up * e_slope[seg // 2] + 1e-6 * g.abs()).all())
    assert bool((dlogp[y == IGN] == 0).all())
    return loss, dlogp, chosen, rejected, ws


@pytest.mark.parametrize("lengths", [[1, 1], [5, 0], [0, 0], [3, 7, 64, 33], [200, 150] * 16, [4097, 3, 1, 5000], [40000, 25000],
                                     [1, 2, 3, 4] * 300])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("length_normalize", [False, True])
def test_preference(cuda_device, lengths, kind, length_normalize):
    start, tail = (7, 5) if len(lengths) % 4 == 0 else (0, 0)
    T = sum(lengths) + start + tail
    logp, _, ref, _, y, g = draw(max(T, 1), cuda_device, seed=T + len(lengths), mask=0.3)
    logp, ref, y = logp[:T].contiguous(), (logp + 0.1 * torch.randn(max(T, 1), generator=g, device=cuda_device))[:T].contiguous(), y[:T].contiguous()
    cu = cu_of(lengths, cuda_device, start)
    P = len(lengths) // 2
    for red in ("mean", "sum", "none"):
        kw = dict(kind=kind, length_normalize=length_normalize, reduction=red, beta=0.3)
        if kind == "sigmoid":
            kw.update(label_smoothing=0.1, margin=0.2)
        if kind == "hinge":
            kw.update(margin=0.05)
        dloss = torch.randn(P if red == "none" else 1, generator=g, device=cuda_device)
        a = check_preference(logp, ref, y, cu, dloss=dloss, longest=max(lengths), **kw)
        b = flce.flce_preference_loss(logp, y, cu, ref_logp=ref, dloss=dloss, workspace=a[-1], **kw)
        assert torch.equal(a[1], b[1]) and torch.equal(a[0], b[0])
    check_preference(logp, None, y, cu, longest=max(lengths), kind=kind, length_normalize=True, beta=2.0)


def test_preference_masked_places_and_large_margins(cuda_device):
    lengths = [300, 200, 50, 0, 10, 10]
    T = sum(lengths)
    logp, _, ref, _, y, _ = draw(T, cuda_device, seed=2)
    y[500:550] = IGN  # a chosen answer without a valid token, and its rejected one is empty
    cu = cu_of(lengths, cuda_device)
    a = check_preference(logp, ref, y, cu, longest=300)
    bad, bad_ref = logp.clone(), ref.clone()
    bad[y == IGN], bad_ref[y == IGN] = float("nan"), float("inf")
    b = flce.flce_preference_loss(bad, y, cu, ref_logp=bad_ref)
    assert all(torch.equal(x, z) for x, z in zip(a[:4], b[:4]))
    assert float(flce.flce_preference_loss(logp, y, cu, ref_logp=ref, reduction="none")[0][1]) == pytest.approx(math.log(2))
    # |h| of hundreds: finite, the softplus linear on one side and zero on the other
    far = logp.clone()
    far[:300] += 1000.0
    loss, dlogp, _, _, _ = flce.flce_preference_loss(far, y, cu, ref_logp=ref, reduction="none")
    assert float(loss[0]) == 0.0 and bool((dlogp[:500] == 0).all())
    far[:300] -= 2000.0
    check_preference(far, ref, y, cu, longest=300)


def test_preference_autograd_and_differences(cuda_device):
    lengths = [60, 40, 30, 80, 25, 25]
    logp, _, ref, _, y, g = draw(sum(lengths), cuda_device, seed=4)
    cu = cu_of(lengths, cuda_device)
    for kw in (dict(label_smoothing=0.1), dict(kind="ipo", length_normalize=True), dict(kind="hinge", beta=0.05)):
        x = logp.clone().requires_grad_(True)
        loss, chosen, rejected = flce.preference_loss(x, y, cu, ref, **kw)
        (3 * loss).backward()
        assert not chosen.requires_grad
        v = torch.randn(logp.numel(), generator=g, device=cuda_device).double()
        step = 1e-5
        value = lambda lp: float(preference_reference(lp, ref, y, cu, **kw)[0])
        want = 3 * (value(logp.double() + step * v) - value(logp.double() - step * v)) / (2 * step)
        assert abs(float((x.grad.double() * v).sum()) - want) <= 1e-5 * float((x.grad.double() * v).abs().sum())


def test_preference_bad_sequences_and_no_pairs(cuda_device):
    logp, _, ref, _, y, _ = draw(100, cuda_device)
    for cu in ([0, 50, 40], [0, 50, 101], [-5, 50, 100], [2 ** 40, 2 ** 41, 3]):
        *_, ws = flce.flce_preference_loss(logp, y, torch.tensor(cu, dtype=torch.int64, device=cuda_device))
        assert flce.flce_read_device_status(ws) == 8
    loss, dlogp, chosen, _, ws = flce.flce_preference_loss(logp, y, torch.zeros(1, dtype=torch.int64, device=cuda_device))
    assert float(loss) == 0 and bool((dlogp == 0).all()) and chosen.numel() == 0 and flce.flce_read_device_status(ws) == 0


def test_preference_refusals(cuda_device):
    logp, _, ref, _, y, _ = draw(16, cuda_device)
    cu = cu_of([8, 8], cuda_device)
    f = flce.flce_preference_loss
    for bad in (dict(beta=0.0), dict(beta=float("inf")), dict(label_smoothing=0.5), dict(label_smoothing=0.1, kind="ipo"),
                dict(margin=0.1, kind="ipo"), dict(margin=float("nan")), dict(forward=False, grad=False)):
        with pytest.raises(flce.FlceError) as e:
            f(logp, y, cu, **bad)
        assert e.value.status == 1, bad
    for args in ((logp.cpu(), y, cu), (logp, y[:8], cu), (logp, y, cu[:2]), (logp, y, cu.int()), (logp.double(), y, cu)):
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(KeyError):
        f(logp, y, cu, reduction="sequence_mean")
    with pytest.raises(flce.FlceError) as e:
        f(logp, y, cu, workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device))
    assert e.value.status == 4
