"""Edges of the operators around the head: long runs of empty sequences, streams of other devices, values beside a
tie, digits near zero, gradients off 16 bytes, second derivatives, device status, scales and values at the ends of their range."""

import pytest
import torch

import lm_head_linear_gb300 as flce

from test_gpu_linear_fp8 import value, whole
from test_gpu_losses import check_policy, draw
from test_gpu_norm import BF, F32

pytestmark = pytest.mark.gpu


def milliseconds(f):
    f()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("T", [4000, 50000])
def test_policy_across_many_empty_sequences(cuda_device, T):
    """300,000 empty sequences between two tokens of one thread: the same values, and no thread
    walks past them one by one (at 0.4 us each that took 120 ms)."""
    logp, old, ref, adv, y, g = draw(T, cuda_device, seed=11)
    n = 300_000
    cu = torch.cat([torch.tensor([0, 1, 1, 7], device=cuda_device), torch.full((n,), 2002, device=cuda_device),
                    torch.tensor([2003, 2003, 3001, T], device=cuda_device)])
    advs = torch.randn(cu.numel() - 1, generator=g, device=cuda_device)
    for red in ("sequence_mean", "mean"):
        kw = dict(reduction=red, kl_coef=0.05, kl="k2")
        check_policy((logp, old, ref, advs, y), dict(kw, cu=cu, per_sequence=True), cu_seqlens=cu, per_sequence=True, **kw)
        call = lambda: flce.flce_policy_loss(logp, old, advs, y, ref_logp=ref, cu_seqlens=cu, per_sequence=True, **kw)
        assert milliseconds(call) < 10.0


class OtherDevice:
    """What a stream of another device looks like (its handle is the current one: nothing can go wrong on it)."""
    device = torch.device("cuda", 1)

    def __init__(self):
        self.cuda_stream = torch.cuda.current_stream().cuda_stream


def test_a_stream_of_another_device_is_refused(cuda_device):
    x = torch.randn(4, 128, device=cuda_device)
    w = torch.ones(128, device=cuda_device)
    logp, old, _, adv, y, _ = draw(16, cuda_device)
    cu = torch.tensor([0, 8, 16], device=cuda_device)
    _, h, rstd, q, qs = flce.flce_add_rms_norm(x, w, fp8=True, save_rstd=True, stream=torch.cuda.current_stream())
    Wq, Ws = flce.flce_quantize_fp8(x)
    s = OtherDevice()
    for call in (lambda: flce.flce_add_rms_norm(x, w, stream=s), lambda: flce.flce_add_rms_norm_backward(x, h, w, rstd, stream=s),
                 lambda: flce.flce_quantize_fp8(x, stream=s), lambda: flce.flce_linear_fp8(q, qs, Wq, Ws, stream=s),
                 lambda: flce.flce_policy_loss(logp, old, adv, y, stream=s),
                 lambda: flce.flce_preference_loss(logp, y, cu, stream=s)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    assert torch.cuda.current_device() == cuda_device.index


@pytest.mark.parametrize("block_rows", [2 ** 32 + 128, 2 ** 32 + 1, -2 ** 32 + 128, 0, -1, 127, 2 ** 31])
def test_quantize_refuses_block_sizes_that_only_look_right_in_32_bits(cuda_device, block_rows):
    """Taken as 128 they would have the kernel write more scales than were allocated."""
    with pytest.raises(flce.FlceError) as e:
        flce.flce_quantize_fp8(torch.randn(512, 128, device=cuda_device), block_rows=block_rows)
    assert e.value.status == 1


def nearest_e4m3(v):
    """|v| <= 448 in 64 bits to the nearest e4m3 number, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    return torch.round(v / step) * step


@pytest.mark.parametrize("x_dtype", [BF, F32])
@pytest.mark.parametrize("T,Hd", [(2, 128), (200, 512), (5000, 512)])
def test_products_beside_a_tie_where_rstd_is_a_power_of_two(cuda_device, x_dtype, T, Hd):
    """rstd is 1 and h w lies off the middle of two e4m3 numbers by less than fp32 resolves: rounded
    once, it goes to the nearer one (no tolerance)."""
    u = 2.0 ** -23
    if x_dtype == BF:
        h = torch.full((Hd,), 0.5, device=cuda_device)
        h[:Hd * 3 // 8] = 1.5           # mean square 1
    else:
        k = torch.arange(Hd // 2, device=cuda_device) % 4 + 1
        h = torch.cat([1 + k * u, 1 - k * u])  # squares 1 +- 2 k u and less than u / 2
    middle = 1 + (2 * (torch.arange(Hd, device=cuda_device) % 8).double() + 1) / 16
    w = (middle / h.double()).float()
    w = torch.where(torch.arange(Hd, device=cuda_device) % 3 == 0, torch.nextafter(w, 2 * w), w)
    y = h.double() * w.double()
    off = y - middle
    assert float(off.abs().max()) < 4 * u and int((off != 0).sum()) > Hd // 2
    x = h.expand(T, Hd).to(x_dtype).contiguous()
    _, _, rstd, q, qs = flce.flce_add_rms_norm(x, w, eps=0.0, normed=False, fp8=True, save_rstd=True)
    assert bool((rstd == 1).all())
    s = torch.ldexp(torch.ones((), dtype=torch.float64, device=cuda_device), qs.view(torch.uint8).int() - 127)
    s = s.repeat_interleave(128, 1)
    assert torch.equal(q.double(), nearest_e4m3(y / s))


@pytest.mark.parametrize("T", [4001, 40001])
def test_k3_keeps_its_digits_near_zero(cuda_device, T):
    """e^e - 1 - e from e = 10^-7 to 8 in both signs.  Bound: below 1/2 the sum of the series, five roundings of at
    most 2^-24; above, one unit in the last place of expm1 (at most 2^-23 of it) against a value that is at least
    0.22 of it, and the subtraction's rounding: below 12 x 2^-24 in either case."""
    size = torch.logspace(-7, 0.9, T // 2, device=cuda_device)
    ref = torch.cat([size, -size, torch.zeros(1, device=cuda_device)])
    zero = torch.zeros(T, device=cuda_device)
    y = torch.ones(T, dtype=torch.int64, device=cuda_device)
    kw = dict(ref_logp=ref, kl_coef=1.0, kl="k3")
    loss, dlogp, _, _, _ = flce.flce_policy_loss(zero, zero, zero, y, reduction="none", **kw)
    e = ref.double()
    want = torch.expm1(e) - e
    assert bool(((loss.double() - want).abs() <= 12 * 2.0 ** -24 * want).all())
    assert bool(((dlogp.double() + torch.expm1(e)).abs() <= 2 ** -22 * torch.expm1(e).abs()).all())
    near = torch.full((T,), 3e-6, device=cuda_device)  # a policy that has hardly moved: the mean over tokens
    stats = flce.flce_policy_loss(zero, zero, zero, y, **dict(kw, ref_logp=near))[2]
    e = near.double()[0]
    assert float(stats[0]) == pytest.approx(float(e * e / 2 + e * e * e / 6), rel=1e-6)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_gradients_off_16_bytes(cuda_device, dtype):
    """Contiguous upstream gradients that start one element into a buffer (slices of a flat one)."""
    T, Hd = 6, 64
    x = torch.randn(T, Hd, device=cuda_device).to(dtype).requires_grad_(True)
    w = torch.rand(Hd, device=cuda_device).requires_grad_(True)
    flat = [torch.randn(1 + T * Hd, device=cuda_device).to(t)[1:] for t in (BF, dtype)]
    dy, dh = (f.view(T, Hd) for f in flat)
    got, want = [], []
    for grads, into in (((dy, dh), got), ((dy.clone(), dh.clone()), want)):
        y, h = flce.add_rms_norm(x, w)
        into += torch.autograd.grad([y, h], [x, w], grads)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_second_derivatives_raise(cuda_device):
    """A gradient that went through an operator is no constant: differentiating it says so.  A gradient of
    the residual sum alone is linear, and has its second derivative."""
    logp, old, ref, adv, y, _ = draw(64, cuda_device, mask=0.0)
    cu = torch.tensor([0, 20, 64], device=cuda_device)
    lp = logp.clone().requires_grad_(True)
    x = torch.randn(8, 64, device=cuda_device).to(BF).requires_grad_(True)
    w = torch.ones(64, device=cuda_device).requires_grad_(True)
    r = torch.randn(8, 64, device=cuda_device).to(BF).requires_grad_(True)
    W = torch.randn(100, 64, device=cuda_device).to(BF).requires_grad_(True)
    yh = torch.arange(8, device=cuda_device)
    for loss, wrt in ((flce.policy_loss(lp, old, adv, y, ref, kl_coef=0.1)[0], lp),
                      (flce.preference_loss(lp, y, cu, ref)[0], lp),
                      (flce.add_rms_norm(x, w, r)[0].float().square().sum(), r),
                      (flce.add_rms_norm(x, w)[0].float().sum(), w),
                      (flce.linear_cross_entropy(x, W, yh), x)):
        plain, = torch.autograd.grad(loss, wrt, retain_graph=True)
        g, = torch.autograd.grad(loss, wrt, create_graph=True)
        assert torch.equal(g, plain) and not plain.requires_grad
        with pytest.raises(RuntimeError, match="first derivatives only"):
            (g * wrt).sum().backward()
    h = flce.add_rms_norm(x, w, r)[1]
    g, = torch.autograd.grad(h.float().pow(3).sum(), x, create_graph=True)
    second, = torch.autograd.grad(g.float().sum(), r)
    assert torch.allclose(second.float(), 6 * h.detach().float(), rtol=2.0 ** -7)


def test_status_of_the_differentiable_losses(cuda_device):
    """With a workspace of the caller's, malformed sequences are known after the forward and after the backward."""
    logp, old, ref, adv, y, _ = draw(100, cuda_device)
    for policy in (True, False):
        n = flce.flce_policy_loss_workspace_size(100, 2) if policy else flce.flce_preference_loss_workspace_size(1)
        for cu, want in (([0, 60, 40], 8), ([0, 60, 100], 0)):
            cu = torch.tensor(cu, device=cuda_device)
            ws = torch.full((n,), 255, dtype=torch.uint8, device=cuda_device)
            x = logp.clone().requires_grad_(True)
            if policy:
                loss = flce.policy_loss(x, old, adv, y, ref, cu, workspace=ws, reduction="sequence_mean")[0]
            else:
                loss = flce.preference_loss(x, y, cu, ref, workspace=ws)[0]
            assert flce.flce_read_device_status(ws) == want
            ws.fill_(255)
            loss.backward()
            assert flce.flce_read_device_status(ws) == want


@pytest.mark.parametrize("T,V", [(1, 300), (40, 600), (240, 700), (600, 257)])
def test_scale_bytes_at_the_ends_of_their_range(cuda_device, T, V):
    """Byte 0 is 2^-127, 254 is 2^127, and 255 a NaN that reaches its own row (or 128 columns) and nothing else."""
    K = 384
    x, sx, W, sw = whole(T, K, V, cuda_device, seed=V)
    for j, (a, b) in enumerate(((0, 254), (254, 0), (127, 127))):
        sx[:, j], sw[:, j] = a, b
    want = x.double() @ W.double().t()  # every block's scales multiply to 1
    y, ws = flce.flce_linear_fp8(x, sx, W, sw, dtype=F32)
    assert torch.equal(y.double(), want)
    rows, blocks = [T // 2], [0, (V - 1) // 128]  # the last one reaches past V
    sx, sw = torch.full_like(sx, 127), torch.full_like(sw, 127)
    sx[rows, 1] = 255
    sw[blocks[0], 2], sw[blocks[1], 0] = 255, 255
    for dtype in (F32, BF):
        y, ws = flce.flce_linear_fp8(x, sx, W, sw, dtype=dtype, workspace=ws)
        assert flce.flce_read_device_status(ws) == 0
        nan = torch.zeros(T, V, dtype=torch.bool, device=cuda_device)
        nan[rows] = True
        for b in blocks:
            nan[:, 128 * b:128 * b + 128] = True
        assert torch.equal(torch.isnan(y), nan)
        assert torch.equal(y[~nan], want.to(dtype)[~nan])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_of_zeros_nan_and_infinities(cuda_device, dtype, block_rows):
    """A block of zeros has the least scale; a NaN stays one and leaves its block's scale alone; an infinity
    saturates at the scale of the largest finite numbers."""
    R, K = 300, 400
    a = torch.randn(R, K, device=cuda_device).to(dtype)
    a[128:256, 128:256] = 0
    a[0, 0] = 0
    a[5, 300] = float("nan")
    a[6, 256:384] = float("nan")
    a[260, 3], a[260, 4] = float("inf"), -float("inf")
    q, s = flce.flce_quantize_fp8(a, block_rows=block_rows)
    clean = a.clone()
    clean[torch.isnan(a)] = 0
    q0, s0 = flce.flce_quantize_fp8(clean, block_rows=block_rows)
    U8 = torch.uint8
    assert torch.equal(s.view(U8), s0.view(U8))
    assert torch.equal(torch.isnan(q.float()), torch.isnan(a))
    assert torch.equal(q.float()[~torch.isnan(a)], q0.float()[~torch.isnan(a)])
    per = 128 // block_rows  # rows of scales for 128 of the matrix
    assert bool((s.view(U8)[per:2 * per, 1] == 1).all()) and bool((q.float()[128:256, 128:256] == 0).all())
    at = 260 if block_rows == 1 else 2
    assert int(s.view(U8)[at, 0]) == 247 and q.float()[260, 3] == 448 and q.float()[260, 4] == -448
    rest = slice(260, 261) if block_rows == 1 else slice(256, 300)
    assert int((q.float()[rest, :128] != 0).sum()) == 2  # what 2^120 leaves of the others


@pytest.mark.parametrize("T,K,V", [(1, 128, 9), (3, 288, 75), (40, 144, 4097), (224, 16, 33), (225, 64, 859), (300, 144, 2),
                                   (400, 304, 4588), (600, 1008, 167), (512, 128, 1030), (130, 128, 255)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_into_columns_of_a_wider_buffer(cuda_device, T, K, V, dtype):
    """Rows on 16 bytes that end inside 16 bytes (one shard's columns of a buffer that holds all): what lies
    before, between and behind the rows keeps its values."""
    x, sx, W, sw = whole(T, K, V, cuda_device, seed=V)
    want = (value(x, sx, 1) @ value(W, sw, 128).t()).float().to(dtype)
    per = 16 // want.element_size()
    for ld in (-(-V // per) * per, (-(-V // per) + 3) * per):
        buf = torch.full((T, ld), 7.0, dtype=dtype, device=cuda_device)
        _, ws = flce.flce_linear_fp8(x, sx, W, sw, dtype=dtype, out={"y": buf[:, :V]})
        assert flce.flce_read_device_status(ws) == 0
        assert torch.equal(buf[:, :V], want)
        assert bool((buf[:, V:] == 7.0).all())
