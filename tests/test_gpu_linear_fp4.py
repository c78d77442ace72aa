"""The head product with 4-bit weights and their quantiser against 64-bit formulas.

Bounds.  Products of e4m3 and e2m1 numbers are exact in fp32 and power-of-two scales add
no error; what rounds is the fp32 accumulation, one step per 32 channels of K:
(K / 32 + 2) steps of at most 2^-22 of the sum of magnitudes.  On inputs whose
partial sums are whole multiples of one power of two below 2^24 of it nothing
rounds at all, and the fp32 output has to be equal.  The quantiser rounds once, and its
numbers have to be equal.
"""

import math

import pytest
import torch

import lm_head_linear_gb300 as flce
from test_gpu_guards import Guarded
from test_gpu_linear_fp8 import value
from test_gpu_norm import half_step_bf16

pytestmark = pytest.mark.gpu

BF, F32, U8, E8 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e8m0fnu
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
POW2 = [math.ldexp(1.0, i - 127) for i in range(255)] + [math.nan]  # of a scale byte (torch.ldexp on a GPU is off by a bit)
SHAPES = [(1, 16, 1), (1, 128, 256), (32, 128, 256), (33, 144, 300), (64, 512, 512), (65, 640, 129), (1, 2048, 4096), (17, 1040, 4097),
          (128, 4096, 1000), (192, 256, 513), (193, 384, 640), (224, 256, 513), (300, 512, 4097), (1000, 1168, 2047), (449, 2048, 20000),
          (256, 128, 8), (512, 640, 232), (1024, 272, 4104), (2000, 1040, 1000), (1, 4112, 30001), (90, 1168, 20011),
          (256, 256, 1), (511, 144, 33), (513, 400, 4099), (768, 272, 1026), (700, 128, 900), (150, 256, 2050)]


def pow2(e):
    return torch.tensor(POW2, dtype=torch.float64, device=e.device)[e.view(U8).long()]


def value4(q, s, K):
    """What packed numbers and their scales stand for, in 64 bits."""
    V, kb = q.shape[0], s.shape[0]
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=q.device)
    codes = torch.stack([q & 15, q >> 4], dim=2).view(V, 128 * kb)
    return (table[codes.long()].view(V, kb, 4, 32) * pow2(s).permute(1, 0, 2)[:, :, :, None]).reshape(V, 128 * kb)[:, :K]


def whole4(T, K, V, dev, seed=0):
    """Operands in {-1, 0, 1}, scales 2^-2 .. 2^2, drawn for every block (of x) and group (of W) on its own."""
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, device=dev)
    kb = -(-K // 128)
    x = r(-1, 2, T, K).float().to(torch.float8_e4m3fn)
    code = torch.tensor([10, 0, 2], dtype=U8, device=dev)[r(0, 3, V, kb * 128)]
    code[:, K:] = 0
    code = code.view(V, kb * 64, 2)
    return x, r(125, 130, T, kb).to(U8), code[:, :, 0] | code[:, :, 1] << 4, r(125, 130, kb, V, 4).to(U8)


@pytest.mark.parametrize("T,K,V", SHAPES)
def test_exact_products(cuda_device, T, K, V):
    x, sx, W, sw = whole4(T, K, V, cuda_device, seed=T + K + V)
    want = value(x, sx, 1) @ value4(W, sw, K).t()
    y, ws = flce.flce_linear_fp4(x, sx, W, sw, dtype=F32)
    assert flce.flce_read_device_status(ws) == 0
    assert torch.equal(y.double(), want)
    y16, _ = flce.flce_linear_fp4(x, sx, W, sw, workspace=ws)
    assert torch.equal(y16, want.float().to(BF))


@pytest.mark.parametrize("T,K,V", SHAPES)
def test_real_operands(cuda_device, T, K, V):
    g = torch.Generator(device=cuda_device).manual_seed(T)
    a = torch.randn(T, K, generator=g, device=cuda_device)
    a[:, ::61] *= 30
    b = torch.randn(V, K, generator=g, device=cuda_device) * 0.02
    x, sx = flce.flce_quantize_fp8(a, block_rows=1)
    W, sw = flce.flce_quantize_fp4(b.to(BF))
    X64, W64 = value(x, sx, 1), value4(W, sw, K)
    want, mag = X64 @ W64.t(), X64.abs() @ W64.abs().t()
    bound = (K / 32 + 2) * 2.0 ** -22 * mag
    y, ws = flce.flce_linear_fp4(x, sx, W, sw, dtype=F32)
    assert bool(((y.double() - want).abs() <= bound).all())
    y16, _ = flce.flce_linear_fp4(x, sx, W, sw, workspace=ws)
    assert bool(((y16.double() - want).abs() <= bound + half_step_bf16(want) * 1.01).all())
    again, _ = flce.flce_linear_fp4(x, sx, W, sw, dtype=F32, workspace=ws)
    assert torch.equal(y, again) and flce.flce_read_device_status(ws) == 0


def test_every_code_and_scale(cuda_device):
    """Each of the 16 numbers under each scale byte that its products stay fp32 numbers for, one number to a group."""
    codes = torch.arange(16, device=cuda_device)
    scales = torch.arange(1, 251, device=cuda_device)
    V = 16 * 250
    W = torch.zeros(V, 64, dtype=U8, device=cuda_device)
    sw = torch.full((1, V, 4), 127, dtype=U8, device=cuda_device)
    row = torch.arange(V, device=cuda_device)
    at = row % 128  # any channel
    W[row, at // 2] = (codes[row % 16] << (4 * (at % 2))).to(U8)
    sw[0, row, at // 32] = scales[row // 16].to(U8)
    x = torch.ones(3, 128, device=cuda_device).to(torch.float8_e4m3fn)
    sx = torch.full((3, 1), 127, dtype=U8, device=cuda_device)
    want = value(x, sx, 1) @ value4(W, sw, 128).t()
    y, _ = flce.flce_linear_fp4(x, sx, W, sw, dtype=F32)
    normal = want.abs() >= 2.0 ** -126  # below, the tensor cores may give zeros
    assert torch.equal(torch.where(normal, y.double(), 0.0), torch.where(normal, want, 0.0))
    assert bool((y.abs() <= 2.0 ** -126)[~normal].all())


def test_strided_output_scale_alignment_and_streams(cuda_device):
    T, K, V = 50, 512, 700
    x, sx, W, sw = whole4(T, K, V, cuda_device, seed=7)
    want = (value(x, sx, 1) @ value4(W, sw, K).t()).float()
    for pad in (0, 1, 3, 64):
        for dtype in (BF, F32):
            wide = torch.full((T, V + pad), 5.0, dtype=dtype, device=cuda_device)
            flce.flce_linear_fp4(x, sx, W, sw, dtype=dtype, out={"y": wide[:, :V]})
            assert torch.equal(wide[:, :V], want.to(dtype)) and bool((wide[:, V:] == 5.0).all())
    raw = torch.zeros(sx.numel() + 1, dtype=U8, device=cuda_device)  # the tokens' scales off a word boundary
    raw[1:] = sx.flatten()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = flce.flce_linear_fp4(x, raw[1:].view(sx.shape), W, sw.view(E8), dtype=F32, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    e = torch.empty(0, K, dtype=torch.float8_e4m3fn, device=cuda_device)
    y, ws = flce.flce_linear_fp4(e, torch.empty(0, 4, dtype=U8, device=cuda_device), W, sw)
    assert y.shape == (0, V) and flce.flce_read_device_status(ws) == 0


@pytest.mark.parametrize("T,K,V", [(1, 144, 257), (3, 256, 131), (70, 256, 1000), (300, 384, 515), (520, 128, 1032)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_guards(cuda_device, T, K, V, dtype):
    x, sx, W, sw = whole4(T, K, V, cuda_device)
    want = (value(x, sx, 1) @ value4(W, sw, K).t()).to(dtype)
    ws, y = Guarded((256,), U8, cuda_device), Guarded((T, V), dtype, cuda_device)
    flce.flce_linear_fp4(x, sx, W, sw, dtype=dtype, workspace=ws.t, out={"y": y.t})
    assert torch.equal(y.t, want) and y.intact() and ws.intact()
    buf = torch.full((T * V + 2001,), 9.0, dtype=dtype, device=cuda_device)  # rows on odd addresses
    at = buf[1001:1001 + T * V].view(T, V)
    flce.flce_linear_fp4(x, sx, W, sw, dtype=dtype, out={"y": at})
    assert torch.equal(at, want) and bool((buf[:1001] == 9.0).all()) and bool((buf[1001 + T * V:] == 9.0).all())
    kb = -(-K // 128)
    q, s = Guarded((V, 64 * kb), U8, cuda_device), Guarded((kb, V, 4), E8, cuda_device)
    flce.flce_quantize_fp4(torch.randn(V, K, device=cuda_device), out={"q": q.t, "q_scale": s.t})
    assert q.intact() and s.intact()


def test_nan_reaches_only_its_own_outputs(cuda_device):
    T, K, V = 40, 256, 600
    x, sx, W, sw = whole4(T, K, V, cuda_device, seed=1)
    want = (value(x, sx, 1) @ value4(W, sw, K).t()).float()
    x8, sw = x.view(U8).clone(), sw.clone()
    x8[7, 200] = 0x7f
    sw[1, 333, 2] = 255  # a group's scale is NaN
    y, _ = flce.flce_linear_fp4(x8.view(torch.float8_e4m3fn), sx, W, sw, dtype=F32)
    assert bool(torch.isnan(y[7]).all()) and bool(torch.isnan(y[:, 333]).all())
    y[7], want[7], y[:, 333], want[:, 333] = 0, 0, 0, 0
    assert torch.equal(y, want)


def check_fp4(q, s, a):
    """a in 64 bits.  The scale rule, and each number the nearest one, ties to the even code."""
    R, K = a.shape
    kb = -(-K // 128)
    assert q.shape == (R, 64 * kb) and s.shape == (kb, R, 4)
    full = torch.nn.functional.pad(a, (0, 128 * kb - K))
    e = s.view(U8).permute(1, 0, 2).reshape(R, 4 * kb)
    sv = pow2(e)
    groups = full.view(R, 4 * kb, 32)
    amax = groups.abs().amax(2)
    assert bool(((amax <= 6 * sv) | (e == 252)).all()) and bool(((amax > 3 * sv) | (e == 1)).all())
    codes = torch.stack([q & 15, q >> 4], dim=2).view(R, 4 * kb, 32)
    v = (groups / sv[:, :, None]).abs().clamp(max=6.0)
    table = torch.tensor(E2M1, dtype=torch.float64, device=a.device)
    mid = (table[1:] + table[:-1]) / 2
    want = torch.bucketize(v, mid)
    for i, m in enumerate(mid.tolist()):  # a tie goes to the even one of codes i and i + 1
        want = torch.where(v == m, i + i % 2, want)
    assert torch.equal((codes & 7).long(), want)
    assert bool((((codes >> 3) == 1) == torch.signbit(groups)).all())


@pytest.mark.parametrize("R,K", [(1, 16), (128, 128), (129, 144), (300, 2048), (1000, 272)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize(cuda_device, R, K, dtype):
    g = torch.Generator(device=cuda_device).manual_seed(R + K)
    a = (torch.randn(R, K + 16, generator=g, device=cuda_device) * torch.exp(3 * torch.randn(R, 1, generator=g, device=cuda_device))).to(dtype)[:, :K]
    check_fp4(*flce.flce_quantize_fp4(a), a.double())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_ties_and_extremes(cuda_device, dtype):
    """Whole quarters of the scale (every tie), the least and the largest numbers, zeros, infinities, NaN."""
    a = torch.zeros(12, 128, device=cuda_device)
    a[0] = torch.arange(-64, 64, device=cuda_device) / 4
    a[1, :64] = torch.arange(0, 64, device=cuda_device) * 2.0 ** -8
    a[2] = 2.0 ** -126
    a[3, ::2], a[3, 1::2] = 2.0 ** -133, -2.0 ** -126
    a[4, :] = 3.0e38
    a[5, 3] = torch.finfo(dtype).max
    a[6, 40] = -0.0
    a[7] = 6.0
    a[8] = 6.0 + 2.0 ** -5
    a[9, 70], a[9, 71] = float("inf"), 1.0
    a[10, 100] = float("nan")
    a[11, 0], a[11, 33] = float("-inf"), float("nan")
    a = a.to(dtype)
    q, s = flce.flce_quantize_fp4(a)
    finite = [0, 1, 2, 3, 4, 5, 6, 7, 8]
    check_fp4(q[finite], s.view(U8)[:, finite].contiguous(), a[finite].double())
    raw = s.view(U8)[0]
    got = value4(q, s, 128)
    assert got[9, 70] == 6 * 2.0 ** 125 and got[9, 71] == 0 and raw[9].tolist() == [1, 1, 252, 1]
    assert raw[10].tolist() == [1, 1, 1, 255] and bool((got[10, :96] == 0).all())
    assert raw[11].tolist() == [252, 255, 1, 1] and got[11, 0] == -6 * 2.0 ** 125


def test_refusals(cuda_device):
    x, sx, W, sw = whole4(4, 256, 300, cuda_device)
    f = flce.flce_linear_fp4
    for args in ((x.float(), sx, W, sw), (x, sx[:, :1], W, sw), (x, sx, W, sw[:1]), (x, sx, W[:, :64], sw), (x, sx, W, sw.int()),
                 (x.cpu(), sx, W, sw), (x, sx, W.to(torch.int8), sw), (x, sx, W, sw.transpose(0, 1)), (x, sx, W[:200], sw)):
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(ValueError):
        f(x, sx, W, sw, dtype=torch.float16)
    with pytest.raises(ValueError):
        f(x, sx, W, sw, out={"y": torch.empty(4, 299, dtype=BF, device=cuda_device)})
    for size, status in ((8, 3), (16, 3)):  # W off 32 bytes
        off = torch.zeros(300 * 128 + 64, dtype=U8, device=cuda_device)[size:size + 300 * 128].view(300, 128)
        with pytest.raises(flce.FlceError) as e:
            f(x, sx, off, sw)
        assert e.value.status == status
    off = torch.zeros(2 * 300 * 4 + 4, dtype=U8, device=cuda_device)[2:2 + 2400].view(2, 300, 4)
    with pytest.raises(flce.FlceError) as e:
        f(x, sx, W, off)
    assert e.value.status == 3
    x8, s8, W8, t8 = whole4(4, 24, 300, cuda_device)
    with pytest.raises(flce.FlceError) as e:
        f(x8, s8, W8, t8)
    assert e.value.status == 2  # K not a multiple of 16
    with pytest.raises(flce.FlceError) as e:
        f(x, sx, W, sw, workspace=torch.empty(128, dtype=U8, device=cuda_device))
    assert e.value.status == 4
    with pytest.raises(flce.FlceError) as e:
        flce.flce_quantize_fp4(torch.zeros(4, 40, device=cuda_device))
    assert e.value.status == 2
    with pytest.raises(ValueError):
        flce.flce_quantize_fp4(torch.zeros(4, 32, device=cuda_device, dtype=torch.float16))


@pytest.mark.parametrize("T,K,V", [(193, 128, 33), (256, 16, 447), (300, 144, 4097), (513, 272, 1111), (700, 640, 9001)])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (2, 1), (3, 2), (5, 4), (7, 9), (0, 6)])
def test_rows_of_any_alignment(cuda_device, T, K, V, offset, pad):
    """bf16 rows that start `offset` elements into a buffer and lie V + pad apart: exact values, and nothing
    written before, between or behind the rows."""
    x, sx, W, sw = whole4(T, K, V, cuda_device, seed=T + V + offset)
    want = (value(x, sx, 1) @ value4(W, sw, K).t()).float().to(BF)
    buf = torch.full((T * (V + pad) + 64,), 7.0, dtype=BF, device=cuda_device)
    y = torch.as_strided(buf, (T, V), (V + pad, 1), 16 + offset)
    out, ws = flce.flce_linear_fp4(x, sx, W, sw, out={"y": y})
    assert flce.flce_read_device_status(ws) == 0
    assert torch.equal(y, want)
    y.fill_(7.0)
    assert bool((buf == 7.0).all())
