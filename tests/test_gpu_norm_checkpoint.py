"""The norm whose backward reads h in 8 bits, against 64-bit formulas and the norm that keeps h.

Bounds.  The forward's y, h and rstd have to be the other norm's bit for bit, and hq is rounded once: its numbers
have to be equal.  The backward is the other norm's arithmetic on the numbers that hq stands for, so its bounds are
test_gpu_norm's: 1e-5 of the sum of magnitudes, and half a step of bf16 where dx is that.
"""

import math

import pytest
import torch

import lm_head_linear_gb300 as flce
from test_gpu_guards import Guarded
from test_gpu_norm import BF, EPS, F32, SHAPES, half_step_bf16, make

pytestmark = pytest.mark.gpu

U8, E4, E8 = torch.uint8, torch.float8_e4m3fn, torch.float8_e8m0fnu
POW2 = [math.ldexp(1.0, i - 127) for i in range(255)] + [math.nan]


def scales(qs, Hd):
    t = torch.tensor(POW2, dtype=torch.float64, device=qs.device)[qs.view(U8).long()]
    return t.repeat_interleave(128, 1)[:, :Hd]


def kept(q, qs):
    return q.double() * scales(qs, q.shape[1])


def check_kept(q, qs, h):
    """The scale rule and the one rounding, of h in 64 bits (finite)."""
    T, Hd = h.shape
    nb = -(-Hd // 128)
    assert q.dtype == E4 and q.shape == (T, Hd) and qs.dtype == E8 and qs.shape == (T, nb)
    amax = torch.nn.functional.pad(h.abs(), (0, nb * 128 - Hd)).view(T, nb, 128).amax(2)
    s = torch.tensor(POW2, dtype=torch.float64, device=h.device)[qs.view(U8).long()]
    assert bool((amax <= 448 * s).all()) and bool(((amax > 224 * s) | (qs.view(U8) == 1)).all())
    v = h / scales(qs, Hd)
    step = torch.where(v.abs() < 2.0 ** -6, 2.0 ** -9, torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3))
    assert torch.equal(q.double(), torch.round(v / step) * step)


def gradient(dy, h64, w, rstd, dh):
    """dx, dweight, and the sums of magnitudes they are made of."""
    r, u, dy64 = rstd.double()[:, None], dy.double() * w.double(), dy.double()
    mean, size = (u * h64).mean(1, keepdim=True), (u * h64).abs().mean(1, keepdim=True)
    dx, mag = r * (u - h64 * r ** 2 * mean), r * (u.abs() + h64.abs() * r ** 2 * size)
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    terms = dy64 * h64 * r
    return dx, mag, terms.sum(0), terms.abs().sum(0)


@pytest.mark.parametrize("T,Hd", SHAPES)
@pytest.mark.parametrize("x_dtype,r_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32), (BF, None), (F32, None)])
def test_forward(cuda_device, T, Hd, x_dtype, r_dtype):
    x, w, r, _ = make(T, Hd, x_dtype, r_dtype, cuda_device, seed=T + Hd, w_dtype=F32 if T % 2 else BF, pad=0 if T % 3 else 16)
    y, h, rstd, q, qs = flce.flce_add_rms_norm_checkpoint(x, w, residual=r, eps=EPS)
    y2, h2, rstd2, _, _ = flce.flce_add_rms_norm(x, w, residual=r, eps=EPS, save_rstd=True)
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(rstd, rstd2) and h.dtype == h2.dtype
    check_kept(q, qs, h.double())


@pytest.mark.parametrize("T,Hd", SHAPES + [(5000, 512)])
@pytest.mark.parametrize("h_dtype,dy_dtype,with_dh", [(BF, BF, True), (F32, BF, False), (F32, F32, True), (BF, F32, False)])
def test_backward(cuda_device, T, Hd, h_dtype, dy_dtype, with_dh):
    h, w, _, g = make(T, Hd, h_dtype, None, cuda_device, seed=T * 3 + Hd, pad=16, w_dtype=F32 if T % 2 else BF)
    dy = torch.randn(T, Hd + 16, generator=g, device=cuda_device).to(dy_dtype)[:, :Hd]
    dh = torch.randn(T, Hd + 16, generator=g, device=cuda_device).to(h_dtype)[:, :Hd] if with_dh else None
    _, _, rstd, q, qs = flce.flce_add_rms_norm_checkpoint(h, w)
    dx, dw, ws = flce.flce_add_rms_norm_checkpoint_backward(dy, q, qs, w, rstd, dh=dh, dtype=h_dtype)
    assert flce.flce_read_device_status(ws) == 0 and dx.dtype == h_dtype
    want, size, dw_want, dw_size = gradient(dy, kept(q, qs), w, rstd, dh)
    assert bool(((dx.double() - want).abs() <= 1e-5 * size + (half_step_bf16(want) * (1 + 1e-9) if h_dtype == BF else 0)).all())
    assert bool(((dw.double() - dw_want).abs() <= 2e-5 * dw_size).all())
    dx2, dw2, _ = flce.flce_add_rms_norm_checkpoint_backward(dy, q, qs.view(U8), w, rstd, dh=dh, dtype=h_dtype, workspace=ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def representable(T, Hd, dev, seed):
    """h that 8 bits hold exactly: whole numbers of four bits times a power of two for each block."""
    g = torch.Generator(device=dev).manual_seed(seed)
    nb = -(-Hd // 128)
    m = torch.randint(-15, 16, (T, nb, 128), generator=g, device=dev).float()
    m *= torch.exp2(torch.randint(-4, 4, (T, nb, 1), generator=g, device=dev).float())
    return m.view(T, nb * 128)[:, :Hd].contiguous(), g


@pytest.mark.parametrize("T,Hd", [(3, 64), (40, 272), (700, 2048), (170, 4112)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_same_gradients_where_eight_bits_hold_h(cuda_device, T, Hd, dtype):
    h, g = representable(T, Hd, cuda_device, T)
    w = (1 + 0.2 * torch.randn(Hd, generator=g, device=cuda_device)).to(BF)
    dy = torch.randn(T, Hd, generator=g, device=cuda_device).to(BF)
    dh = torch.randn(T, Hd, generator=g, device=cuda_device).to(dtype)
    grads = []
    for checkpoint in (False, True):
        x, r, wg = h.to(dtype).requires_grad_(True), torch.zeros_like(h, dtype=dtype).requires_grad_(True), w.clone().requires_grad_(True)
        y, hh = flce.add_rms_norm(x, wg, r, EPS, checkpoint=checkpoint)
        assert torch.equal(hh, h.to(dtype))
        torch.autograd.backward([y, hh], [dy, dh])
        grads.append((y.detach(), x.grad, r.grad, wg.grad))
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_gradient_against_differences(cuda_device):
    """Where 8 bits hold h, the gradient is the norm's: central differences of sum(y dy) + sum(h dh) in 64 bits."""
    T, Hd = 6, 96
    h, g = representable(T, Hd, cuda_device, 1)
    w = 1 + 0.2 * torch.randn(Hd, generator=g, device=cuda_device)
    dy = torch.randn(T, Hd, generator=g, device=cuda_device).to(BF)
    dh = torch.randn(T, Hd, generator=g, device=cuda_device)
    xg, wg = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    y, hh = flce.add_rms_norm(xg, wg, eps=EPS, checkpoint=True)
    torch.autograd.backward([y, hh], [dy, dh])
    dy64, dh64 = dy.double(), dh.double()

    def loss(x64, w64):
        y64 = x64 / torch.sqrt((x64 * x64).mean(1, keepdim=True) + EPS) * w64
        return float((y64 * dy64).sum() + (x64 * dh64).sum())

    base = [h.double(), w.double()]
    for i, grad in enumerate((xg.grad, wg.grad)):
        v = torch.randn(base[i].shape, generator=g, device=cuda_device).double()
        step = 1e-4
        hi = [b + (step * v if k == i else 0) for k, b in enumerate(base)]
        lo = [b - (step * v if k == i else 0) for k, b in enumerate(base)]
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        assert abs(float((grad.double() * v).sum()) - want) <= 1e-5 * float((grad.double() * v).abs().sum())


def test_what_the_graph_holds(cuda_device):
    T, Hd = 300, 1040
    x, w, r, _ = make(T, Hd, BF, BF, cuda_device)
    xg, rg = x.requires_grad_(True), r.requires_grad_(True)
    y, h = flce.add_rms_norm(xg, w, rg, checkpoint=True)
    held = {(tuple(t.shape), t.dtype) for t in y.grad_fn.saved_tensors}
    assert held == {((T, Hd), E4), ((T, 9), E8), ((Hd,), BF), ((T,), F32)}
    del h
    y.float().sum().backward()  # dh is not there; dy an expanded tensor
    assert xg.grad.shape == x.shape and torch.equal(xg.grad, rg.grad)
    only_h = flce.add_rms_norm(xg, w, rg, checkpoint=True)[1]
    xg.grad = None
    only_h.float().sum().backward()
    assert bool((xg.grad == 1).all())
    with pytest.raises(RuntimeError):
        y, _ = flce.add_rms_norm(xg, w, rg, checkpoint=True)
        (d,) = torch.autograd.grad(y.float().sum(), xg, create_graph=True)
        d.float().sum().backward()


def test_extreme_rows(cuda_device):
    T, Hd = 8, 384
    x = torch.randn(T, Hd, device=cuda_device)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[3, 200] = float("nan")
    x[4, 5] = float("inf")
    x[5, 128:256] = 0
    x[6, ::2] *= 2.0 ** -40  # far below its block's scale
    w = torch.ones(Hd, device=cuda_device)
    y, _, rstd, q, qs = flce.flce_add_rms_norm_checkpoint(x, w)
    y2, _, rstd2, _, _ = flce.flce_add_rms_norm(x, w, save_rstd=True)
    same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), 1e9), torch.nan_to_num(b.float(), 1e9))
    assert same(y, y2) and same(rstd, rstd2)
    ok = [0, 1, 2, 5, 6, 7]
    check_kept(q[ok], qs.view(U8)[ok].view(E8), x[ok].double())
    assert bool((q[0].float() == 0).all()) and bool((qs.view(U8)[0] == 1).all())
    assert bool(torch.isnan(q[3, 200].float())) and int(torch.isnan(q[3].float()).sum()) == 1
    dy = torch.randn(T, Hd, device=cuda_device)
    dx, dw, _ = flce.flce_add_rms_norm_checkpoint_backward(dy, q, qs, w, rstd, dtype=F32)
    want, size, _, _ = gradient(dy, kept(q, qs), w, rstd, None)
    assert bool(((dx.double() - want).abs() <= 1e-5 * size)[ok].all())
    assert bool(torch.isnan(dx[3]).all()) and bool(torch.isnan(dw[200]))


@pytest.mark.parametrize("T,Hd", [(1, 16), (3, 144), (301, 2064), (700, 4112)])
def test_guards_in_place_and_graph(cuda_device, T, Hd):
    x, w, r, _ = make(T, Hd, BF, F32, cuda_device, w_dtype=F32)
    nb = -(-Hd // 128)
    fwd = {"h": ((T, Hd), F32), "y": ((T, Hd), BF), "rstd": ((T,), F32), "hq": ((T, Hd), E4), "hq_scale": ((T, nb), E8)}
    bwd = {"dx": ((T, Hd), F32), "dweight": ((Hd,), F32)}
    g1, g2 = ({k: Guarded(s, t, cuda_device) for k, (s, t) in d.items()} for d in (fwd, bwd))
    o1, o2 = ({k: v.t for k, v in d.items()} for d in (g1, g2))
    ws = Guarded((flce.flce_add_rms_norm_backward_workspace_size(T, Hd),), U8, cuda_device)

    def step():
        flce.flce_add_rms_norm_checkpoint(x, w, residual=r, out=o1)
        flce.flce_add_rms_norm_checkpoint_backward(x, o1["hq"], o1["hq_scale"], w, o1["rstd"], dh=r, dtype=F32, workspace=ws.t, out=o2)

    step()
    assert all(v.intact() for v in (*g1.values(), *g2.values(), ws))
    want = {k: v.clone() for k, v in (o1 | o2).items()}
    r2 = r.clone()
    h = flce.flce_add_rms_norm_checkpoint(x, w, residual=r2, out={"h": r2})[1]
    assert h.data_ptr() == r2.data_ptr() and torch.equal(r2, want["h"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in (o1 | o2).values():
        v.view(U8).zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(v.view(U8), want[k].view(U8)) for k, v in (o1 | o2).items())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = flce.flce_add_rms_norm_checkpoint(x, w, residual=r, stream=s)[0]
    s.synchronize()
    assert torch.equal(y, want["y"])


def test_no_rows_and_refusals(cuda_device):
    w = torch.ones(64, device=cuda_device)
    x = torch.empty(0, 64, dtype=BF, device=cuda_device)
    y, h, rstd, q, qs = flce.flce_add_rms_norm_checkpoint(x, w, residual=x)
    assert y.shape == (0, 64) and qs.shape == (0, 1)
    dx, dw, ws = flce.flce_add_rms_norm_checkpoint_backward(x, q, qs, w, rstd)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and flce.flce_read_device_status(ws) == 0
    x, w, r, _ = make(4, 128, BF, BF, cuda_device)
    f, b = flce.flce_add_rms_norm_checkpoint, flce.flce_add_rms_norm_checkpoint_backward
    for args in ((x.cpu(), w), (x.half(), w), (x, w[:64]), (x, w, r[:2])):
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(flce.FlceError) as e:
        f(x[:, :120], w[:120].contiguous())
    assert e.value.status == 2
    y, h, rstd, q, qs = f(x, w, residual=r)
    for args in ((x, q.view(U8), qs, w, rstd), (x, q, qs[:2], w, rstd), (x, q, qs, w, rstd.double()), (x, q, qs, w, rstd, r.float()),
                 (x[:2], q, qs, w, rstd), (x, q.float(), qs, w, rstd), (x, q[:, :64], qs, w, rstd)):
        with pytest.raises(ValueError):
            b(*args)
    with pytest.raises(ValueError):
        b(x, q, qs, w, rstd, dtype=torch.float16)
    with pytest.raises(flce.FlceError) as e:
        b(x, q, qs, w, rstd, workspace=torch.empty(256, dtype=U8, device=cuda_device))
    assert e.value.status == 4
