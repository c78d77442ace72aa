"""The operators of a rollout and its training step together, and what they have in common with the others: the
chain as a program runs it, captured graphs, two streams, launches dispatched early, a bounded wait that runs out,
offsets past 32 bits, the timing aid, and the example with them."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import lm_head_linear_gb300 as flce
from test_gpu_linear_fp4 import value4, whole4
from test_gpu_linear_fp8 import value
from test_gpu_sample import draw_row

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
E4 = torch.float8_e4m3fn
IGN = -100


def state(dev, seed, S=24, Hd=512, V=5003):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *n: torch.randn(*n, generator=g, device=dev)
    s = {"x": r(S, Hd).to(BF), "r": r(S, Hd).to(BF), "w": 0.5 + torch.rand(Hd, generator=g, device=dev), "W": (r(V, Hd) * 0.2).to(BF),
         "u": torch.rand(S, generator=g, device=dev), "k": torch.randint(0, 3000, (S,), generator=g, device=dev).int(),
         "dy": r(S, Hd).to(BF)}
    s["Wq"], s["Ws"] = flce.flce_quantize_fp4(s["W"])
    s["ws"] = [torch.empty(n, dtype=U8, device=dev) for n in (256, flce.flce_add_rms_norm_backward_workspace_size(S, Hd))]
    return s


def step(s):
    """A decoding step, and a norm kept in 8 bits with its backward."""
    _, h, _, q, qs = flce.flce_add_rms_norm(s["x"], s["w"], residual=s["r"], normed=False, fp8=True)
    logits, _ = flce.flce_linear_fp4(q, qs, s["Wq"], s["Ws"], dtype=F32, workspace=s["ws"][0])
    tokens, logp = flce.flce_sample(logits, s["u"], temperature=0.9, top_k=s["k"], top_p=0.95, min_p=0.001)
    y, h2, rstd, hq, hs = flce.flce_add_rms_norm_checkpoint(s["x"], s["w"], residual=s["r"])
    dx, dw, _ = flce.flce_add_rms_norm_checkpoint_backward(s["dy"], hq, hs, s["w"], rstd, workspace=s["ws"][1])
    return [h, q.view(U8), qs.view(U8), logits, tokens, logp, y, h2, rstd, hq.view(U8), hs.view(U8), dx, dw]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_decoding_step(cuda_device):
    """Norm to 8 bits, product with 4-bit weights, draw: each from the definition on what the one before gave."""
    s = state(cuda_device, 1)
    out = step(s)
    q, qs, logits, tokens, logp = out[1].view(E4), out[2], out[3], out[4], out[5]
    X, W = value(q, qs, 1), value4(s["Wq"], s["Ws"], 512)
    want, mag = X @ W.t(), X.abs() @ W.abs().t()
    assert bool(((logits.double() - want).abs() <= (512 / 32 + 2) * 2.0 ** -22 * mag).all())
    for i in range(24):
        t, lp = draw_row(logits[i].double().cpu().numpy(), float(s["u"][i]), 0.9, int(s["k"][i]), 0.95, 0.001)
        assert int(tokens[i]) == t and abs(float(logp[i]) - lp) <= 2.0 ** -24 * abs(lp) + 2.0 ** -24 + 2.0 ** -29
    assert flce.flce_read_device_status(s["ws"][0]) == 0 and flce.flce_read_device_status(s["ws"][1]) == 0
    # the token and its logp are what the losses take: a row that a mask leaves empty is ignored there
    logits[3] = float("-inf")
    tokens, logp = flce.flce_sample(logits, s["u"], ignore_index=IGN)
    loss, dlogp, _, n, _ = flce.flce_policy_loss(logp, logp, torch.ones(24, device=cuda_device), tokens, ignore_index=IGN)
    assert int(n) == 23 and float(dlogp[3]) == 0 and abs(float(loss) + 1) <= 2.0 ** -20


def test_training_through_the_checkpoint(cuda_device):
    """Norm, head and loss by autograd, the norm's input kept in 8 bits: the gradients are the low-level calls' one by one."""
    T, Hd, V = 96, 128, 500
    g = torch.Generator(device=cuda_device).manual_seed(3)
    x, r = (torch.randn(T, Hd, generator=g, device=cuda_device).to(BF).requires_grad_(True) for _ in range(2))
    w = (torch.rand(Hd, generator=g, device=cuda_device) + 0.5).requires_grad_(True)
    W = (torch.randn(V, Hd, generator=g, device=cuda_device) * 0.1).to(BF).requires_grad_(True)
    y = torch.randint(0, V, (T,), generator=g, device=cuda_device)
    y[::5] = IGN
    adv = torch.randn(T, generator=g, device=cuda_device)
    old = -6 + 0.3 * torch.randn(T, generator=g, device=cuda_device)
    h, res = flce.add_rms_norm(x, w, r, checkpoint=True)
    logp = flce.linear_log_probs(h, W, y, IGN)
    loss, _ = flce.policy_loss(logp, old, adv, y, kl_coef=0.0)
    (loss + 1e-3 * res.float().sum()).backward()
    n, hh, rstd, hq, hs = flce.flce_add_rms_norm_checkpoint(x.detach(), w.detach(), residual=r.detach())
    h2 = n.clone().requires_grad_(True)
    W2 = W.detach().clone().requires_grad_(True)
    flce.policy_loss(flce.linear_log_probs(h2, W2, y, IGN), old, adv, y, kl_coef=0.0)[0].backward()
    dh = torch.full_like(hh, 1e-3)
    dx, dw, _ = flce.flce_add_rms_norm_checkpoint_backward(h2.grad, hq, hs, w.detach(), rstd, dh=dh)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dx) and torch.equal(w.grad, dw) and torch.equal(W.grad, W2.grad)
    # and near the gradients of the norm that keeps h: an element of the checkpoint is off by at most 2^-4 of it or
    # 2^-10 of its block's scale; the terms that h enters are a small part of dx and the errors have no sign in common
    x2, r2, w2 = (t.detach().clone().requires_grad_(True) for t in (x, r, w))
    flce.add_rms_norm(x2, w2, r2)[0].backward(h2.grad)
    assert float((x2.grad.double() - (dx.double() - dh.double())).norm() / x2.grad.double().norm()) <= 2.0 ** -4
    assert float((w2.grad.double() - dw.double()).norm() / dw.double().norm()) <= 2.0 ** -4


def test_graph_replays_on_new_inputs(cuda_device):
    s, other = state(cuda_device, 1), state(cuda_device, 2)
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s)
    for k in ("x", "r", "w", "u", "k", "dy", "Wq"):
        s[k].copy_(other[k])
    s["Ws"].view(U8).copy_(other["Ws"].view(U8))
    for _ in range(2):
        for t in got:
            t.view(U8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, step(other))


def test_two_streams_at_once(cuda_device):
    states = [state(cuda_device, 3), state(cuda_device, 4, S=3, V=70001)]
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
    """A rollout in which every step's tokens choose the next step's inputs, call by call and in one go."""
    s = state(cuda_device, 7)
    embed = torch.randn(5003, 512, device=cuda_device).to(BF)

    def rollout(wait):
        x, r, tokens = s["x"], s["r"], []
        for _ in range(10):
            _, r, _, q, qs = flce.flce_add_rms_norm(x, s["w"], residual=r, normed=False, fp8=True)
            if wait:
                torch.cuda.synchronize()
            logits, _ = flce.flce_linear_fp4(q, qs, s["Wq"], s["Ws"], workspace=s["ws"][0])
            if wait:
                torch.cuda.synchronize()
            t, _ = flce.flce_sample(logits, s["u"], top_p=0.9)
            if wait:
                torch.cuda.synchronize()
            tokens.append(t)
            x = embed[t]
        return torch.stack(tokens)

    want = rollout(True)
    for _ in range(5):
        assert torch.equal(rollout(False), want)


def test_abort_path_of_the_4_bit_product(cuda_device):
    """As the 8-bit product's: a K of 4,194,304 and a limit of 1 ms; FLCE_ERR_TIMEOUT, the context stays usable, and
    with the default limit the product is right."""
    K, V = 4194304, 256
    W = torch.full((V, K // 2), 0x22, dtype=U8, device=cuda_device)  # ones
    W[1:] = 0x20
    sw = torch.full((K // 128, V, 4), 125, dtype=U8, device=cuda_device)
    for T in (2, 200):
        x = torch.ones(T, K, device=cuda_device).to(E4)
        sx = torch.full((T, K // 128), 120, dtype=U8, device=cuda_device)
        try:
            flce.flce_set_wait_timeout_ns(1_000_000)
            _, ws = flce.flce_linear_fp4(x, sx, W, sw, dtype=F32)
            assert flce.flce_read_device_status(ws) == 7
        finally:
            flce.flce_set_wait_timeout_ns(4_000_000_000)
        y, ws = flce.flce_linear_fp4(x, sx, W, sw, dtype=F32, workspace=ws)
        assert flce.flce_read_device_status(ws) == 0
        scale = 2.0 ** (120 + 125 - 254)
        assert bool((y[:, 0] == K * scale).all()) and bool((y[:, 1:] == K / 2 * scale).all())


def test_offsets_past_32_bits(cuda_device):
    T, K, V = 17500, 64, 248320  # 4.3e9 logits
    x, sx, W, sw = whole4(T, K, V, cuda_device, seed=9)
    y, ws = flce.flce_linear_fp4(x, sx, W, sw)
    assert flce.flce_read_device_status(ws) == 0
    rows = [0, 1, 127, 128, 8191, 12287, 17248, 17407, 17499]
    want = value(x, sx, 1)[rows] @ value4(W, sw, K).t()
    assert torch.equal(y[rows].double(), want.float().to(BF).double())
    u = torch.rand(T, device=cuda_device)
    t, lp = flce.flce_sample(y, u, top_p=0.5)
    few, lp_few = flce.flce_sample(y[rows], u[rows], top_p=0.5)
    assert torch.equal(t[rows], few) and torch.equal(lp[rows], lp_few)
    del y
    V, K = 34000, 327680  # and past them in W: 5.6e9 bytes
    W = torch.randint(0, 256, (V, K // 2), dtype=U8, device=cuda_device) & 0x33  # 0, 0.5, 1, 1.5
    sw = torch.full((K // 128, V, 4), 127, dtype=U8, device=cuda_device)
    x = torch.randint(-1, 2, (3, K), device=cuda_device).float().to(E4)
    sx = torch.full((3, K // 128), 127, dtype=U8, device=cuda_device)
    y, ws = flce.flce_linear_fp4(x, sx, W, sw, dtype=F32)
    assert flce.flce_read_device_status(ws) == 0
    at = [0, 63, 64, 13107, 13108, 26214, 32768, 33999]
    assert torch.equal(y[:, at].double(), x.double() @ value4(W[at].contiguous(), sw[:, at].contiguous(), K).t())
    a = torch.zeros(V, K, dtype=BF, device=cuda_device)  # 1.1e10 elements quantised
    a[at] = torch.randn(len(at), K, device=cuda_device).to(BF)
    q, s = flce.flce_quantize_fp4(a)
    few = flce.flce_quantize_fp4(a[at])
    assert torch.equal(q[at], few[0]) and torch.equal(s.view(U8)[:, at], few[1].view(U8))


def test_checkpoint_offsets_past_32_bits(cuda_device):
    T, Hd = 530000, 8192  # 4.3e9 elements
    w = torch.ones(Hd, device=cuda_device)
    x = torch.empty(T, Hd, dtype=BF, device=cuda_device)
    for a in range(0, T, 53000):
        x[a:a + 53000] = torch.randn(1, Hd, device=cuda_device).to(BF) * (1 + a / 53000)
    y, _, rstd, hq, hs = flce.flce_add_rms_norm_checkpoint(x, w)
    dx, dw, ws = flce.flce_add_rms_norm_checkpoint_backward(y, hq, hs, w, rstd, dh=x)
    assert flce.flce_read_device_status(ws) == 0
    for part in (slice(0, 3000), slice(262100, 265100), slice(527000, 530000)):
        few = flce.flce_add_rms_norm_checkpoint(x[part], w)
        assert torch.equal(y[part], few[0]) and torch.equal(hq[part].view(U8), few[3].view(U8)) and torch.equal(hs[part].view(U8), few[4].view(U8))
        d = flce.flce_add_rms_norm_checkpoint_backward(y[part], hq[part], hs[part], w, rstd[part], dh=x[part])[0]
        assert torch.equal(dx[part], d)


def test_timing_aid_names_the_operators(cuda_device):
    s = state(cuda_device, 5)
    step(s)
    flce.flce_profile_collect()
    flce.flce_profile_enable(True)
    try:
        step(s)
        flce.flce_quantize_fp4(s["W"])
    finally:
        flce.flce_profile_enable(False)
    stats = flce.flce_profile_collect()
    assert {k: v["launches"] for k, v in stats.items()} == {"add_rms_norm": 2, "linear_fp4": 1, "sample": 1, "norm_bwd": 1, "norm_dw": 1,
                                                             "quantize_fp4": 1}
    assert all(v["total_ms"] > 0 for v in stats.values())
    assert stats["linear_fp4"]["flops"] == pytest.approx(2.0 * 24 * 512 * 5003)


@pytest.mark.parametrize("weights", [8, 4])
def test_example_runs(cuda_device, weights):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "rl_step.py")
    spec = importlib.util.spec_from_file_location("rl_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    log = module.run(sequences=6, length=48, hidden=256, vocab=1003, steps=3, seed=2, weights=weights, top_p=0.9, checkpoint=True)
    assert len(log) == 6 and all(np.isfinite(v) for m in log for v in m.values())
