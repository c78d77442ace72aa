"""What the operators around the head have in common: no write outside an output or
a workspace, capture in a CUDA graph, calls on two streams at once, a bounded wait
that runs out, offsets past 32 bits, the timing aid, and the example that chains them."""

import numpy as np
import pytest
import torch

import lm_head_linear_gb300 as flce

from test_gpu_guards import Guarded
from test_gpu_linear_fp8 import value, whole
from test_gpu_losses import IGN, cu_of, draw

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def outputs(shapes, dev):
    g = {k: Guarded(s, t, dev) for k, (s, t) in shapes.items()}
    return g, {k: v.t for k, v in g.items()}


@pytest.mark.parametrize("T,Hd", [(1, 16), (3, 144), (301, 2064), (700, 4112)])
def test_norm_guards(cuda_device, T, Hd):
    x = torch.randn(T, Hd, device=cuda_device).to(BF)
    r = torch.randn(T, Hd, device=cuda_device)
    w = torch.ones(Hd, device=cuda_device)
    g, out = outputs({"h": ((T, Hd), F32), "y": ((T, Hd), BF), "rstd": ((T,), F32), "q": ((T, Hd), E4),
                      "q_scale": ((T, -(-Hd // 128)), E8)}, cuda_device)
    y, h, rstd, _, _ = flce.flce_add_rms_norm(x, w, residual=r, fp8=True, save_rstd=True, out=out)
    assert all(v.intact() for v in g.values())
    ws = Guarded((flce.flce_add_rms_norm_backward_workspace_size(T, Hd),), U8, cuda_device)
    g, out = outputs({"dx": ((T, Hd), F32), "dweight": ((Hd,), F32)}, cuda_device)
    flce.flce_add_rms_norm_backward(x, h, w, rstd, dh=r, workspace=ws.t, out=out)
    assert all(v.intact() for v in g.values()) and ws.intact()


@pytest.mark.parametrize("T", [1, 1003, 32769, 70001])
@pytest.mark.parametrize("reduction", ["mean", "none", "sequence_mean"])
def test_policy_guards(cuda_device, T, reduction):
    logp, old, ref, adv, y, _ = draw(T, cuda_device)
    cu = cu_of([T // 3, 0, T - T // 3], cuda_device)
    ws = Guarded((flce.flce_policy_loss_workspace_size(T, 3),), U8, cuda_device)
    g, out = outputs({"loss": ((T if reduction == "none" else 1,), F32), "dlogp": ((T,), F32), "stats": ((4,), F32),
                      "n_valid": ((1,), torch.int64)}, cuda_device)
    flce.flce_policy_loss(logp, old, adv, y, ref_logp=ref, cu_seqlens=cu, reduction=reduction, workspace=ws.t, out=out)
    assert all(v.intact() for v in g.values()) and ws.intact()


@pytest.mark.parametrize("lengths", [[1, 2], [5, 0, 700, 333], [9000, 7001, 1, 4], [40, 50] * 100])
@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_preference_guards(cuda_device, lengths, reduction):
    T, P = sum(lengths), len(lengths) // 2
    logp, _, ref, _, y, _ = draw(T, cuda_device)
    ws = Guarded((flce.flce_preference_loss_workspace_size(P),), U8, cuda_device)
    g, out = outputs({"loss": ((P if reduction == "none" else 1,), F32), "dlogp": ((T,), F32), "chosen": ((P,), F32),
                      "rejected": ((P,), F32)}, cuda_device)
    flce.flce_preference_loss(logp, y, cu_of(lengths, cuda_device), ref_logp=ref, reduction=reduction, workspace=ws.t, out=out)
    assert all(v.intact() for v in g.values()) and ws.intact()


@pytest.mark.parametrize("T,K,V", [(1, 144, 257), (70, 256, 1000), (300, 384, 515), (520, 128, 1032)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_guards(cuda_device, T, K, V, dtype):
    x, sx, W, sw = whole(T, K, V, cuda_device)
    ws = Guarded((256,), U8, cuda_device)
    g, out = outputs({"y": ((T, V), dtype)}, cuda_device)
    flce.flce_linear_fp8(x, sx, W, sw, dtype=dtype, workspace=ws.t, out=out)
    assert g["y"].intact() and ws.intact()
    g, out = outputs({"q": ((V, K), E4), "q_scale": ((-(-V // 128), -(-K // 128)), E8)}, cuda_device)
    flce.flce_quantize_fp8(torch.randn(V, K, device=cuda_device), out=out)
    assert all(v.intact() for v in g.values())


def step(s):
    """Every operator once, on preallocated inputs."""
    y, h, rstd, q, qs = flce.flce_add_rms_norm(s["x"], s["w"], residual=s["r"], fp8=True, save_rstd=True)
    logits, _ = flce.flce_linear_fp8(q, qs, s["Wq"], s["Ws"], workspace=s["ws"][0])
    loss, dlogp, stats, n, _ = flce.flce_policy_loss(s["logp"], s["old"], s["adv"], s["y"], ref_logp=s["ref"],
                                                     cu_seqlens=s["cu"], reduction="sequence_mean", workspace=s["ws"][1])
    ploss, pd, c, r, _ = flce.flce_preference_loss(s["logp"], s["y"], s["cu"], ref_logp=s["ref"], workspace=s["ws"][2])
    dx, dw, _ = flce.flce_add_rms_norm_backward(y, h, s["w"], rstd, dh=s["r"], workspace=s["ws"][3])
    return [h, y, rstd, q, qs, logits, loss, dlogp, stats, n, ploss, pd, c, r, dx, dw]


def state(dev, seed, T=600, tokens=40000):
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"x": torch.randn(T, 512, generator=g, device=dev).to(BF), "r": torch.randn(T, 512, generator=g, device=dev).to(BF),
         "w": torch.rand(512, generator=g, device=dev) + 0.5}
    s["Wq"], s["Ws"] = flce.flce_quantize_fp8(torch.randn(3001, 512, generator=g, device=dev))
    s["logp"], s["old"], s["ref"], s["adv"], s["y"], _ = draw(tokens, dev, seed=seed)
    s["cu"] = cu_of([tokens // 8] * 8, dev)
    s["ws"] = [torch.empty(n, dtype=U8, device=dev) for n in (
        256, flce.flce_policy_loss_workspace_size(tokens, 8), flce.flce_preference_loss_workspace_size(4),
        flce.flce_add_rms_norm_backward_workspace_size(T, 512))]
    return s


def same(a, b):
    return all(torch.equal(x.view(U8) if x.element_size() == 1 else x, y.view(U8) if y.element_size() == 1 else y)
               for x, y in zip(a, b))


@pytest.mark.parametrize("tokens", [20000, 40000])
def test_graph_replays_on_new_inputs(cuda_device, tokens):
    s, other = state(cuda_device, 1, tokens=tokens), state(cuda_device, 2, tokens=tokens)
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s)
    for k in ("x", "r", "w", "logp", "old", "ref", "adv", "y"):
        s[k].copy_(other[k])
    s["Wq"].view(U8).copy_(other["Wq"].view(U8))
    s["Ws"].view(U8).copy_(other["Ws"].view(U8))
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, step(other))


def test_two_streams_at_once(cuda_device):
    states = [state(cuda_device, 3), state(cuda_device, 4)]
    want = [step(s) for s in states]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(states[i])
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_back_to_back_calls_see_each_others_results(cuda_device):
    """Launches may be dispatched before the one ahead of them is done: a chain in
    which every call reads what the last one wrote equals the chain run call by call."""
    T, Hd = 700, 1024
    w = torch.rand(Hd, device=cuda_device) + 0.5
    Wq, Ws = flce.flce_quantize_fp8(torch.randn(Hd, Hd, device=cuda_device) * 0.05)

    def chain(wait):
        x = torch.arange(T * Hd, device=cuda_device).view(T, Hd).remainder(17).sub(8).to(BF)
        r = torch.zeros_like(x)
        for _ in range(12):
            _, r, _, q, qs = flce.flce_add_rms_norm(x, w, residual=r, normed=False, fp8=True)
            if wait:
                torch.cuda.synchronize()
            x, _ = flce.flce_linear_fp8(q, qs, Wq, Ws)
            if wait:
                torch.cuda.synchronize()
        return r

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)


def test_abort_path_of_the_8_bit_product(cuda_device):
    """A K of 4,194,304 keeps a tile's accumulator busy for milliseconds: with the wait
    limit at 1 ms the epilogue gives up inside a legitimate product; the call reports
    FLCE_ERR_TIMEOUT, the context stays usable, and with the default limit it is right."""
    T, K, V = 2, 4194304, 256
    x = torch.ones(T, K, device=cuda_device).to(E4)
    W = torch.ones(V, K, device=cuda_device).to(E4)
    W[1:, ::2] = 0
    sx = torch.full((T, K // 128), 120, dtype=U8, device=cuda_device)
    sw = torch.full((2, K // 128), 125, dtype=U8, device=cuda_device)
    try:
        flce.flce_set_wait_timeout_ns(1_000_000)
        _, ws = flce.flce_linear_fp8(x, sx, W, sw, dtype=F32)
        assert flce.flce_read_device_status(ws) == 7
    finally:
        flce.flce_set_wait_timeout_ns(4_000_000_000)
    y, ws = flce.flce_linear_fp8(x, sx, W, sw, dtype=F32, workspace=ws)
    assert flce.flce_read_device_status(ws) == 0
    scale = 2.0 ** (120 + 125 - 254)
    assert bool((y[:, 0] == K * scale).all()) and bool((y[:, 1:] == K / 2 * scale).all())


def test_linear_offsets_past_32_bits(cuda_device):
    T, K, V = 17500, 64, 248320  # 4.3e9 logits
    x, sx, W, sw = whole(T, K, V, cuda_device, seed=9)
    y, ws = flce.flce_linear_fp8(x, sx, W, sw)
    assert flce.flce_read_device_status(ws) == 0
    rows = [0, 1, 127, 128, 8191, 12287, 17248, 17407, 17499]
    want = value(x, sx, 1)[rows] @ value(W, sw, 128).t()
    assert torch.equal(y[rows].double(), want.float().to(BF).double())
    del y
    V = 17000  # and past them in W: 5.6e9 bytes
    K = 327680
    g = torch.Generator(device=cuda_device).manual_seed(1)
    W = torch.randint(0, 3, (V, K), generator=g, device=cuda_device, dtype=torch.int8).sub_(1).to(E4)
    sw = torch.full((-(-V // 128), K // 128), 127, dtype=U8, device=cuda_device)
    x = torch.randint(-1, 2, (3, K), generator=g, device=cuda_device).float().to(E4)
    sx = torch.full((3, K // 128), 127, dtype=U8, device=cuda_device)
    y, ws = flce.flce_linear_fp8(x, sx, W, sw, dtype=F32)
    assert flce.flce_read_device_status(ws) == 0
    at = [0, 63, 64, 6553, 6554, 13107, 16384, 16999]
    assert torch.equal(y[:, at].double(), x.double() @ W[at].double().t())


def test_norm_offsets_past_32_bits(cuda_device):
    T, Hd = 530000, 8192  # 4.3e9 elements
    w = torch.ones(Hd, device=cuda_device)
    x = torch.empty(T, Hd, dtype=BF, device=cuda_device)
    for a in range(0, T, 53000):
        x[a:a + 53000] = torch.randn(1, Hd, device=cuda_device).to(BF) * (1 + a / 53000)
    y, _, rstd, q, qs = flce.flce_add_rms_norm(x, w, fp8=True, save_rstd=True)
    # the same rows in a call of 3000 (launched in the same shape, so every sum has the same order)
    parts = [slice(0, 3000), slice(262100, 265100), slice(524200, 527200), slice(527000, 530000)]
    for part in parts:
        few = flce.flce_add_rms_norm(x[part], w, fp8=True, save_rstd=True)
        assert torch.equal(y[part], few[0]) and torch.equal(rstd[part], few[2])
        assert torch.equal(q[part].view(U8), few[3].view(U8)) and torch.equal(qs[part].view(U8), few[4].view(U8))
    del q, qs
    dx, dw, ws = flce.flce_add_rms_norm_backward(y, x, w, rstd, dh=x)
    assert flce.flce_read_device_status(ws) == 0
    for part in parts:
        assert torch.equal(dx[part], flce.flce_add_rms_norm_backward(y[part], x[part], w, rstd[part], dh=x[part])[0])


def test_timing_aid_names_the_operators(cuda_device):
    s = state(cuda_device, 5)
    step(s)
    flce.flce_profile_collect()
    flce.flce_profile_enable(True)
    try:
        step(s)
    finally:
        flce.flce_profile_enable(False)
    stats = flce.flce_profile_collect()
    assert set(stats) == {"add_rms_norm", "linear_fp8", "policy_loss", "preference_loss", "norm_bwd", "norm_dw"}
    assert all(v["launches"] == 1 and v["total_ms"] > 0 for v in stats.values())
    assert stats["linear_fp8"]["flops"] == pytest.approx(2.0 * 600 * 512 * 3001)


def test_example_moves_the_policy(cuda_device):
    """The example's chain on a small size: finite figures, and the updates do what the losses ask for."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "rl_step.py")
    spec = importlib.util.spec_from_file_location("rl_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    log = module.run(sequences=8, length=64, hidden=256, vocab=1003, steps=4, seed=1)
    assert all(np.isfinite(v) for m in log for v in m.values())
    policy = [m for m in log if "policy_loss" in m]
    # the first step starts from the rollout policy: ratio 1, no KL, nothing clipped
    assert policy[0]["ratio"] == 1.0 and policy[0]["kl"] == 0.0 and policy[0]["clipped"] == 0.0
    assert policy[-1]["policy_loss"] < policy[0]["policy_loss"]
    prefs = [m for m in log if "preference_loss" in m]
    assert prefs[-1]["preference_loss"] < prefs[0]["preference_loss"] and prefs[-1]["margin"] > prefs[0]["margin"]


def test_chain_gradients_against_plain_autograd(cuda_device):
    """Norm, head, policy loss and back: gradients of the norm's weight, the head and the
    inputs against torch autograd of the same formulas in 64 bits (on the bf16 norm the head sees)."""
    T, Hd, V = 96, 128, 500
    g = torch.Generator(device=cuda_device).manual_seed(3)
    x = torch.randn(T, Hd, generator=g, device=cuda_device).to(BF)
    r = torch.randn(T, Hd, generator=g, device=cuda_device).to(BF)
    w = torch.rand(Hd, generator=g, device=cuda_device) + 0.5
    W = (torch.randn(V, Hd, generator=g, device=cuda_device) * 0.1).to(BF)
    y = torch.randint(0, V, (T,), generator=g, device=cuda_device)
    y[::5] = IGN
    adv = torch.randn(T, generator=g, device=cuda_device)
    old = -6 + 0.3 * torch.randn(T, generator=g, device=cuda_device)
    ins = [t.clone().requires_grad_(True) for t in (x, r, w, W)]
    h, _ = flce.add_rms_norm(ins[0], ins[2], ins[1])
    logp = flce.linear_log_probs(h, ins[3], y, IGN)
    loss, _ = flce.policy_loss(logp, old, adv, y, old + 0.1, kl_coef=0.1, reduction="mean")
    loss.backward()
    # the reference: 64 bits, with the roundings to bf16 that the definitions have (h and the norm) passed straight through
    ref = [t.detach().double().requires_grad_(True) for t in (x, r, w, W)]
    s = ref[0] + ref[1]
    s = s + ((x.float() + r.float()).to(BF).double() - s).detach()
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * ref[2]
    n = n + (h.detach().double() - n).detach()
    z = torch.log_softmax(n @ ref[3].t(), dim=1)
    at = (y != IGN).nonzero()[:, 0]
    lp = z[at, y[at]]
    d = lp - old.double()[at]
    A = adv.double()[at]
    e = old.double()[at] + 0.1 - lp
    per = -torch.minimum(d.exp() * A, d.exp().clamp(0.8, 1.2) * A) + 0.1 * (e.exp() - 1 - e)
    per.mean().backward()
    for got, want in zip(ins, ref):
        assert float((got.grad.double() - want.grad).norm() / want.grad.norm()) <= 1e-2  # the framework's bar for gradients
