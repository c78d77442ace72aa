"""The 8-bit head product and the quantiser against 64-bit formulas.

Bounds.  Products of e4m3 numbers are exact in fp32 and power-of-two scales add
no error; what rounds is the fp32 accumulation, one step per 32 channels of K:
(K / 32 + 2) steps of at most 2^-22 of the sum of magnitudes.  On inputs whose
partial sums are whole multiples of one power of two below 2^24 of it nothing
rounds at all, and the fp32 output has to be equal.
"""

import pytest
import torch

import lm_head_linear_gb300 as flce
from test_gpu_norm import check_fp8, half_step_bf16

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 16, 1), (1, 128, 256), (32, 128, 256), (33, 144, 300), (64, 512, 512), (65, 640, 129), (1, 2048, 4096), (17, 1040, 4097),
          (128, 4096, 1000), (224, 256, 513), (225, 384, 640), (300, 512, 4097), (1000, 1168, 2047), (449, 2048, 20000),
          (256, 128, 8), (512, 640, 232), (1024, 272, 4104), (2000, 1040, 1000),
          (256, 256, 1), (511, 144, 33), (513, 400, 4099), (768, 272, 1026), (700, 128, 900), (150, 256, 2050)]


def value(q, s, rows):
    e = s.view(torch.uint8).int() - 127
    f = torch.ldexp(torch.ones(1, dtype=torch.float64, device=q.device), e)
    return q.double() * f.repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def whole(T, K, V, dev, seed=0):
    """Operands in {-1, 0, 1} with scales 2^-2 .. 2^2, drawn for every block on its own."""
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, device=dev)
    kb = -(-K // 128)
    x = r(-1, 2, T, K).float().to(torch.float8_e4m3fn)
    W = r(-1, 2, V, K).float().to(torch.float8_e4m3fn)
    return x, r(125, 130, T, kb).to(torch.uint8), W, r(125, 130, -(-V // 128), kb).to(torch.uint8)


@pytest.mark.parametrize("T,K,V", SHAPES)
def test_exact_products(cuda_device, T, K, V):
    x, sx, W, sw = whole(T, K, V, cuda_device, seed=T + K + V)
    want = value(x, sx, 1) @ value(W, sw, 128).t()
    y, ws = flce.flce_linear_fp8(x, sx, W, sw, dtype=F32)
    assert flce.flce_read_device_status(ws) == 0
    assert torch.equal(y.double(), want)
    y16, _ = flce.flce_linear_fp8(x, sx, W, sw, workspace=ws)
    assert torch.equal(y16, want.float().to(BF))


@pytest.mark.parametrize("T,K,V", SHAPES)
def test_real_operands(cuda_device, T, K, V):
    g = torch.Generator(device=cuda_device).manual_seed(T)
    a = torch.randn(T, K, generator=g, device=cuda_device)
    a[:, ::61] *= 30
    b = torch.randn(V, K, generator=g, device=cuda_device) * 0.02
    x, sx = flce.flce_quantize_fp8(a, block_rows=1)
    W, sw = flce.flce_quantize_fp8(b.to(BF))
    X64, W64 = value(x, sx, 1), value(W, sw, 128)
    want, mag = X64 @ W64.t(), X64.abs() @ W64.abs().t()
    bound = (K / 32 + 2) * 2.0 ** -22 * mag
    y, ws = flce.flce_linear_fp8(x, sx, W, sw, dtype=F32)
    assert bool(((y.double() - want).abs() <= bound).all())
    y16, _ = flce.flce_linear_fp8(x, sx, W, sw, workspace=ws)
    assert bool(((y16.double() - want).abs() <= bound + half_step_bf16(want) * 1.01).all())
    again, _ = flce.flce_linear_fp8(x, sx, W, sw, dtype=F32, workspace=ws)
    assert torch.equal(y, again) and flce.flce_read_device_status(ws) == 0


def test_strided_output_scale_alignment_and_streams(cuda_device):
    T, K, V = 50, 512, 700
    x, sx, W, sw = whole(T, K, V, cuda_device, seed=7)
    want = (value(x, sx, 1) @ value(W, sw, 128).t()).float()
    for pad in (0, 1, 3, 64):
        for dtype in (BF, F32):
            wide = torch.full((T, V + pad), 5.0, dtype=dtype, device=cuda_device)
            flce.flce_linear_fp8(x, sx, W, sw, dtype=dtype, out={"y": wide[:, :V]})
            assert torch.equal(wide[:, :V], want.to(dtype)) and bool((wide[:, V:] == 5.0).all())
    # scale arrays off a word boundary take the byte path
    raw = torch.zeros(sx.numel() + 1, dtype=torch.uint8, device=cuda_device)
    raw[1:] = sx.flatten()
    raw_w = torch.zeros(sw.numel() + 3, dtype=torch.uint8, device=cuda_device)
    raw_w[3:] = sw.flatten()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = flce.flce_linear_fp8(x, raw[1:].view(sx.shape), W, raw_w[3:].view(sw.shape), dtype=F32, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    e = torch.empty(0, K, dtype=torch.float8_e4m3fn, device=cuda_device)
    y, ws = flce.flce_linear_fp8(e, torch.empty(0, 4, dtype=torch.uint8, device=cuda_device), W, sw)
    assert y.shape == (0, V) and flce.flce_read_device_status(ws) == 0


def test_guards_and_odd_output_alignment(cuda_device):
    """Nothing outside y is written, also where rows start on odd addresses."""
    for T, K, V in ((3, 256, 257), (230, 128, 131), (1, 1024, 4097)):
        x, sx, W, sw = whole(T, K, V, cuda_device, seed=T)
        want = (value(x, sx, 1) @ value(W, sw, 128).t()).float()
        for dtype in (BF, F32):
            buf = torch.full((T * V + 2001,), 9.0, dtype=dtype, device=cuda_device)
            y = buf[1001:1001 + T * V].view(T, V)
            flce.flce_linear_fp8(x, sx, W, sw, dtype=dtype, out={"y": y})
            assert torch.equal(y, want.to(dtype))
            assert bool((buf[:1001] == 9.0).all()) and bool((buf[1001 + T * V:] == 9.0).all())


def test_nan_and_infinite_reach_only_their_own_outputs(cuda_device):
    T, K, V = 40, 256, 600
    x, sx, W, sw = whole(T, K, V, cuda_device, seed=1)
    want = (value(x, sx, 1) @ value(W, sw, 128).t()).float()
    x8, W8 = x.view(torch.uint8).clone(), W.view(torch.uint8).clone()
    x8[7, 200] = 0x7f
    W8[333, 3] = 0xff
    y, _ = flce.flce_linear_fp8(x8.view(torch.float8_e4m3fn), sx, W8.view(torch.float8_e4m3fn), sw, dtype=F32)
    assert bool(torch.isnan(y[7]).all()) and bool(torch.isnan(y[:, 333]).all())
    y[7], want[7], y[:, 333], want[:, 333] = 0, 0, 0, 0
    assert torch.equal(y, want)


@pytest.mark.parametrize("R,K", [(1, 16), (128, 128), (129, 144), (300, 2048), (1000, 272)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize(cuda_device, R, K, dtype):
    g = torch.Generator(device=cuda_device).manual_seed(R + K)
    a = (torch.randn(R, K + 16, generator=g, device=cuda_device) * torch.exp(3 * torch.randn(R, 1, generator=g, device=cuda_device))).to(dtype)[:, :K]
    q, s = flce.flce_quantize_fp8(a, block_rows=1)
    check_fp8(q, s, a.double())
    q, s = flce.flce_quantize_fp8(a)
    nr, nb = -(-R // 128), -(-K // 128)
    assert s.shape == (nr, nb)
    full = torch.zeros(nr * 128, nb * 128, dtype=torch.float64, device=cuda_device)
    full[:R, :K] = a.double()
    amax = full.abs().view(nr, 128, nb, 128).amax((1, 3))
    sv = torch.ldexp(torch.ones(1, dtype=torch.float64, device=cuda_device), s.view(torch.uint8).int() - 127)
    assert bool((amax <= 448 * sv).all()) and bool(((amax > 224 * sv) | (s.view(torch.uint8) == 1)).all())
    v = a.double() / sv.repeat_interleave(128, 0)[:R].repeat_interleave(128, 1)[:, :K]
    assert torch.equal(q.float(), v.float().to(torch.float8_e4m3fn).float())


def test_refusals(cuda_device):
    x, sx, W, sw = whole(4, 256, 300, cuda_device)
    f = flce.flce_linear_fp8
    for args in ((x.float(), sx, W, sw), (x, sx[:, :1], W, sw), (x, sx, W, sw[:2]), (x, sx, W[:, :128], sw), (x, sx.int(), W, sw),
                 (x.cpu(), sx, W, sw)):
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(ValueError):
        f(x, sx, W, sw, dtype=torch.float16)
    with pytest.raises(ValueError):
        f(x, sx, W, sw, out={"y": torch.empty(4, 299, dtype=BF, device=cuda_device)})
    x8, s8, W8, t8 = whole(4, 24, 300, cuda_device)
    with pytest.raises(flce.FlceError) as e:
        f(x8, s8, W8, t8)
    assert e.value.status == 2  # K not a multiple of 16
    off = torch.zeros(4 * 256 + 8, dtype=torch.uint8, device=cuda_device)[8:].view(torch.float8_e4m3fn).view(4, 256)
    with pytest.raises(flce.FlceError) as e:
        f(off, sx, W, sw)
    assert e.value.status == 3
    with pytest.raises(flce.FlceError) as e:
        f(x, sx, W, sw, workspace=torch.empty(128, dtype=torch.uint8, device=cuda_device))
    assert e.value.status == 4
    with pytest.raises(flce.FlceError) as e:
        flce.flce_quantize_fp8(torch.zeros(4, 32, device=cuda_device), block_rows=64)
    assert e.value.status == 1


@pytest.mark.parametrize("T,K,V", [(225, 128, 33), (256, 16, 447), (300, 144, 4097), (513, 272, 1111), (260, 128, 17),
                                   (700, 640, 9001), (2048, 128, 2003)])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (2, 1), (3, 2), (5, 4), (6, 7), (7, 9), (8, 3), (0, 6)])
def test_rows_of_any_alignment(cuda_device, T, K, V, offset, pad):
    """bf16 rows that start `offset` elements into a buffer and lie V + pad apart: exact values, and nothing
    written before, between or behind the rows."""
    x, sx, W, sw = whole(T, K, V, cuda_device, seed=T + V + offset)
    want = (value(x, sx, 1) @ value(W, sw, 128).t()).float().to(BF)
    buf = torch.full((T * (V + pad) + 64,), 7.0, dtype=BF, device=cuda_device)
    y = torch.as_strided(buf, (T, V), (V + pad, 1), 16 + offset)
    out, ws = flce.flce_linear_fp8(x, sx, W, sw, out={"y": y})
    assert flce.flce_read_device_status(ws) == 0
    assert torch.equal(y, want)
    y.fill_(7.0)
    assert bool((buf == 7.0).all())
