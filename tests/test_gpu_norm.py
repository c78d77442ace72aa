"""Residual add + RMS norm, its 8-bit output and its backward, against 64-bit formulas.

Bounds.  A row's sum of squares is at most 72 fp32 additions deep (up to 64
values on a thread, then a tree), so rstd is within 40 * 2^-24 and an fp32 y
within 48 * 2^-24 < 3e-6 of the exact one, relatively; bf16 and e4m3 add half a
step of their format at the value.
"""

import pytest
import torch

import lm_head_linear_gb300 as flce

pytestmark = pytest.mark.gpu

EPS = 1e-6
REL = 3e-6          # fp32 part of y's error
SHAPES = [(1, 16), (1, 2048), (3, 64), (5, 128), (7, 144), (2, 4112), (33, 1040), (300, 2048), (161, 4096), (1000, 256),
          (2, 16384), (157, 16384), (513, 8208)]
BF, F32 = torch.bfloat16, torch.float32


def half_step_bf16(v):
    """Half the distance of bf16 numbers at |v| (8 significant bits)."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -126))) - 8)


def make(T, Hd, x_dtype, r_dtype, dev, seed=0, pad=0, w_dtype=BF):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(T, Hd + pad, generator=g, device=dev)
    x[:, ::37] *= 20.0
    w = (1 + 0.2 * torch.randn(Hd, generator=g, device=dev)).to(w_dtype)
    r = (2 * torch.randn(T, Hd + pad, generator=g, device=dev)).to(r_dtype)[:, :Hd] if r_dtype is not None else None
    return x.to(x_dtype)[:, :Hd], w, r, g


def reference(x, w, r, eps=EPS):
    """h as the definition rounds it (one fp32 addition, one rounding), the rest in 64 bits."""
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    h64 = h.double()
    rstd = 1 / torch.sqrt((h64 * h64).mean(1) + eps)
    return h, rstd, h64 * rstd[:, None] * w.double()


def check_fp8(q, qs, y):
    T, Hd = y.shape
    nb = -(-Hd // 128)
    assert q.dtype == torch.float8_e4m3fn and qs.shape == (T, nb) and qs.dtype == torch.float8_e8m0fnu
    e = qs.view(torch.uint8).int() - 127
    s = torch.ldexp(torch.ones(1, dtype=torch.float64, device=y.device), e)
    amax = torch.nn.functional.pad(y.abs(), (0, nb * 128 - Hd)).view(T, nb, 128).amax(2)
    assert bool((amax * (1 - REL) <= 448 * s).all())                                    # large enough
    assert bool(((amax * (1 + REL) > 448 * s / 2) | (e == -126)).all())                 # and no larger
    sv = s.repeat_interleave(128, 1)[:, :Hd]
    v = y / sv
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -9))).clamp(min=-6) - 3)
    assert bool(((q.double() - v).abs() <= 0.5 * step * (1 + 1e-9) + 2 * REL * v.abs()).all())


@pytest.mark.parametrize("T,Hd", SHAPES)
@pytest.mark.parametrize("x_dtype,r_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32), (BF, None), (F32, None)])
def test_forward(cuda_device, T, Hd, x_dtype, r_dtype):
    x, w, r, _ = make(T, Hd, x_dtype, r_dtype, cuda_device, seed=T + Hd, w_dtype=F32 if T % 2 else BF)
    y, h, rstd, q, qs = flce.flce_add_rms_norm(x, w, residual=r, eps=EPS, fp8=True, save_rstd=True)
    h_ref, rstd_ref, y_ref = reference(x, w, r)
    assert torch.equal(h, h_ref) and h.dtype == h_ref.dtype
    assert bool(((rstd.double() - rstd_ref).abs() <= REL * rstd_ref).all())
    assert bool(((y.double() - y_ref).abs() <= half_step_bf16(y_ref) * (1 + 1e-9) + 2 * REL * y_ref.abs()).all())
    check_fp8(q, qs, y_ref)


@pytest.mark.parametrize("T,Hd", [(1, 2048), (77, 1040), (400, 4096)])
def test_outputs_do_not_depend_on_which_are_asked_for_or_on_strides(cuda_device, T, Hd):
    x, w, r, _ = make(T, Hd, BF, BF, cuda_device, pad=64)
    y, h, rstd, q, qs = flce.flce_add_rms_norm(x, w, residual=r, fp8=True, save_rstd=True)
    y2, h2, _, _, _ = flce.flce_add_rms_norm(x.contiguous(), w, residual=r.contiguous())
    _, h3, _, q3, qs3 = flce.flce_add_rms_norm(x, w, residual=r, normed=False, fp8=True)
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(h, h3)
    assert torch.equal(q.view(torch.uint8), q3.view(torch.uint8))
    assert torch.equal(qs.view(torch.uint8), qs3.view(torch.uint8))
    wide = torch.full((T, Hd + 64), 7.0, dtype=BF, device=cuda_device)  # h into a wider buffer; the rest stays
    flce.flce_add_rms_norm(x, w, residual=r, out={"h": wide[:, :Hd]})
    assert torch.equal(wide[:, :Hd], h) and bool((wide[:, Hd:] == 7.0).all())
    r2 = r.clone()                                                     # h written over the residual itself
    y4, h4, _, _, _ = flce.flce_add_rms_norm(x, w, residual=r2, out={"h": r2})
    assert h4.data_ptr() == r2.data_ptr() and torch.equal(r2, h) and torch.equal(y4, y)


def test_extreme_rows(cuda_device):
    """Zero rows, tiny and huge values, one NaN, an infinite entry, blocks of zeros."""
    T, Hd = 9, 384
    x = torch.randn(T, Hd, device=cuda_device)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[3, 200] = float("nan")
    x[4, 5] = float("inf")
    x[5, 128:256] = 0
    x[6] = 0
    x[6, 0] = 1e-4
    w = torch.ones(Hd, device=cuda_device)
    y, _, rstd, q, qs = flce.flce_add_rms_norm(x, w, fp8=True, save_rstd=True)
    ok = [0, 1, 2, 5, 6, 7, 8]
    _, rstd_ref, y_ref = reference(x, w, None)
    assert bool(((rstd.double() - rstd_ref).abs() <= REL * rstd_ref)[ok].all())
    assert bool(((y.double() - y_ref).abs() <= half_step_bf16(y_ref) * (1 + 1e-9) + 2 * REL * y_ref.abs())[ok].all())
    assert bool((q[0].float() == 0).all()) and bool((qs.view(torch.uint8)[0] == 1).all())
    check_fp8(q[[2, 5, 7, 8]], qs[[2, 5, 7, 8]], y_ref[[2, 5, 7, 8]])
    # a NaN anywhere makes its row's sum NaN; an infinity makes rstd 0
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(q[3].float()).all())
    assert rstd[4] == 0 and bool(torch.isnan(y[4, 5])) and bool((y[4, 6:] == 0).all())
    assert bool(torch.isnan(q[4, 5].float())) and bool((q[4, 6:].float() == 0).all())


def test_zero_rows_and_streams(cuda_device):
    w = torch.ones(64, device=cuda_device)
    x = torch.empty(0, 64, dtype=BF, device=cuda_device)
    y, h, rstd, q, qs = flce.flce_add_rms_norm(x, w, residual=x, fp8=True, save_rstd=True)
    assert y.shape == (0, 64) and qs.shape == (0, 1)
    dx, dw, ws = flce.flce_add_rms_norm_backward(x, h, w, rstd)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and flce.flce_read_device_status(ws) == 0
    x, w, r, _ = make(500, 1024, BF, BF, cuda_device)
    want = flce.flce_add_rms_norm(x, w, residual=r)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = flce.flce_add_rms_norm(x, w, residual=r, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,Hd", SHAPES + [(5000, 512)])
@pytest.mark.parametrize("h_dtype,dy_dtype,with_dh", [(BF, BF, True), (F32, BF, False), (F32, F32, True), (BF, F32, False)])
def test_backward(cuda_device, T, Hd, h_dtype, dy_dtype, with_dh):
    h, w, _, g = make(T, Hd, h_dtype, None, cuda_device, seed=T * 3 + Hd, pad=16)
    dy = torch.randn(T, Hd, generator=g, device=cuda_device).to(dy_dtype)
    dh = torch.randn(T, Hd + 16, generator=g, device=cuda_device).to(h_dtype)[:, :Hd] if with_dh else None
    _, _, rstd, _, _ = flce.flce_add_rms_norm(h, w, save_rstd=True)
    dx, dw, ws = flce.flce_add_rms_norm_backward(dy, h, w, rstd, dh=dh)
    assert flce.flce_read_device_status(ws) == 0 and dx.dtype == h_dtype
    h64, dy64 = h.double(), dy.double()
    r = 1 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + EPS)
    u = dy64 * w.double()
    back = h64 * r ** 2 * (u * h64).mean(1, keepdim=True)
    want = r * (u - back) + (dh.double() if with_dh else 0)
    size = r * (u.abs() + h64.abs() * r ** 2 * (u * h64).abs().mean(1, keepdim=True)) + (dh.double().abs() if with_dh else 0)
    assert bool(((dx.double() - want).abs() <= 1e-5 * size + (half_step_bf16(want) * (1 + 1e-9) if h_dtype == BF else 0)).all())
    # dweight: a chain of fewer than 300 fp32 additions per column
    terms = dy64 * h64 * r
    assert bool(((dw.double() - terms.sum(0)).abs() <= 2e-5 * terms.abs().sum(0)).all())
    dx2, dw2, _ = flce.flce_add_rms_norm_backward(dy, h, w, rstd, dh=dh, workspace=ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,Hd", [(1, 16), (5, 144), (700, 2048), (33, 4112), (160, 14336), (160, 14352), (157, 16384)])
@pytest.mark.parametrize("h_dtype,dy_dtype", [(F32, F32), (BF, F32), (F32, BF), (BF, BF)])
def test_backward_with_weights_in_32_bits(cuda_device, T, Hd, h_dtype, dy_dtype):
    """fp32 weights, which for the widest fp32 rows do not fit beside them on chip."""
    h, w, _, g = make(T, Hd, h_dtype, None, cuda_device, seed=T + Hd, w_dtype=F32)
    dy = torch.randn(T, Hd, generator=g, device=cuda_device).to(dy_dtype)
    dh = torch.randn(T, Hd, generator=g, device=cuda_device).to(h_dtype)
    _, _, rstd, _, _ = flce.flce_add_rms_norm(h, w, save_rstd=True)
    dx, dw, ws = flce.flce_add_rms_norm_backward(dy, h, w, rstd, dh=dh)
    assert flce.flce_read_device_status(ws) == 0
    h64, dy64 = h.double(), dy.double()
    r = 1 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + EPS)
    u = dy64 * w.double()
    want = r * (u - h64 * r ** 2 * (u * h64).mean(1, keepdim=True)) + dh.double()
    size = r * (u.abs() + h64.abs() * r ** 2 * (u * h64).abs().mean(1, keepdim=True)) + dh.double().abs()
    assert bool(((dx.double() - want).abs() <= 1e-5 * size + (half_step_bf16(want) * (1 + 1e-9) if h_dtype == BF else 0)).all())
    terms = dy64 * h64 * r
    assert bool(((dw.double() - terms.sum(0)).abs() <= 2e-5 * terms.abs().sum(0)).all())


def test_gradient_against_differences(cuda_device):
    """Directional derivatives of sum(y dy) + sum(h dh) by central differences in 64 bits."""
    T, Hd = 6, 96
    x, w, r, g = make(T, Hd, F32, F32, cuda_device, seed=3, w_dtype=F32)
    xg, wg, rg = (t.clone().requires_grad_(True) for t in (x, w, r))
    dy = torch.randn(T, Hd, generator=g, device=cuda_device)
    dh = torch.randn(T, Hd, generator=g, device=cuda_device)
    y, h = flce.add_rms_norm(xg, wg, rg, eps=EPS)
    torch.autograd.backward([y, h], [dy.to(BF), dh])
    dy64, dh64 = dy.to(BF).double(), dh.double()

    def value(x64, w64, r64):
        h64 = x64 + r64
        y64 = h64 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + EPS) * w64
        return float((y64 * dy64).sum() + (h64 * dh64).sum())

    base = [x.double(), w.double(), r.double()]
    for i, grad in enumerate((xg.grad, wg.grad, rg.grad)):
        v = torch.randn(base[i].shape, generator=g, device=cuda_device).double()
        step = 1e-4
        hi = [b + (step * v if k == i else 0) for k, b in enumerate(base)]
        lo = [b - (step * v if k == i else 0) for k, b in enumerate(base)]
        want = (value(*hi) - value(*lo)) / (2 * step)
        # fp32 gradient, the stored h rounded to fp32, a difference of order step^2
        assert abs(float((grad.double() * v).sum()) - want) <= 1e-5 * float((grad.double() * v).abs().sum())


def test_autograd_without_residual_and_expanded_gradients(cuda_device):
    x, w, _, g = make(20, 256, BF, None, cuda_device)
    xg, wg = x.contiguous().requires_grad_(True), w.clone().requires_grad_(True)
    y, h = flce.add_rms_norm(xg, wg)
    (y.float().sum() + 3 * h.float().sum()).backward()
    _, _, rstd, _, _ = flce.flce_add_rms_norm(x, w, save_rstd=True)
    one = torch.ones_like(x.contiguous())
    dx, dw, _ = flce.flce_add_rms_norm_backward(one, x, w, rstd, dh=3 * one)
    assert torch.equal(xg.grad, dx) and torch.equal(wg.grad, dw.to(BF))
    xg.grad = None
    flce.add_rms_norm(xg, wg)[1].float().sum().backward()  # only h is used
    assert torch.equal(xg.grad, one)


def test_refusals(cuda_device):
    x, w, r, _ = make(4, 128, BF, BF, cuda_device)
    with pytest.raises(ValueError):
        flce.flce_add_rms_norm(x.cpu(), w)
    with pytest.raises(ValueError):
        flce.flce_add_rms_norm(x.half(), w)
    with pytest.raises(ValueError):
        flce.flce_add_rms_norm(x, w[:64])
    with pytest.raises(ValueError):
        flce.flce_add_rms_norm(x, w, residual=r[:2])
    with pytest.raises(ValueError):
        flce.flce_add_rms_norm(x.t().contiguous().t(), w)  # rows not contiguous
    with pytest.raises(flce.FlceError) as e:
        flce.flce_add_rms_norm(x[:, :120], w[:120].contiguous())
    assert e.value.status == 2
    with pytest.raises(flce.FlceError) as e:
        flce.flce_add_rms_norm(x[:, 4:116], w[:112].contiguous())  # base off 16 bytes
    assert e.value.status == 3
    with pytest.raises(flce.FlceError) as e:
        flce.flce_add_rms_norm(x, w, normed=False)
    assert e.value.status == 1
    with pytest.raises(flce.FlceError) as e:
        flce.flce_add_rms_norm(x, w, eps=-1.0)
    assert e.value.status == 1
    _, h, rstd, _, _ = flce.flce_add_rms_norm(x, w, residual=r, save_rstd=True)
    with pytest.raises(ValueError):
        flce.flce_add_rms_norm_backward(x, h, w, rstd.double())
    with pytest.raises(ValueError):
        flce.flce_add_rms_norm_backward(x, h, w, rstd, dh=h.float())
    with pytest.raises(flce.FlceError) as e:
        flce.flce_add_rms_norm_backward(x, h, w, rstd, workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device))
    assert e.value.status == 4
