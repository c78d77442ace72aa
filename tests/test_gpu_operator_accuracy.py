"""The digits that the norm's 8-bit output and the preference loss's sums carry beyond plain fp32.

8 bits: the sum of squares, rstd and the product keep what fp32 rounds off, so an element differs from the 64-bit
definition only where the value lies within about 2^-30 of the middle of two e4m3 numbers, 2^-3 .. 2^-4 apart: about
one in 10^8.  Rounded step by step (2^-23 of the value) it is one in 10^6.  The tests allow 8 x 10^-8 of the elements (and
at least 4 of them): far above the one and far below the other.

Preference rewards: a log ratio is one fp32 subtraction; the sums of the rounded ratios keep what fp32 rounds off
(chains of fp32 corrections: below 2^-40 of the sum of magnitudes for 10^5 tokens) and the reward is rounded once.
"""

import pytest
import torch

import lm_head_linear_gb300 as flce

from test_gpu_losses import IGN, cu_of
from test_gpu_norm import BF, F32
from test_gpu_operator_edges import nearest_e4m3

pytestmark = pytest.mark.gpu


def definition(h, w, eps):
    """(e4m3 values, scale exponents) of rms_norm(h) w in 64 bits."""
    h = h.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double()
    T, Hd = y.shape
    nb = -(-Hd // 128)
    y = torch.nn.functional.pad(y, (0, nb * 128 - Hd)).view(T, nb, 128)
    m, e = torch.frexp(y.abs().amax(2))  # m 2^e, m in [1/2, 1)
    e = (e - 9 + (m > 0.875)).clamp(min=-126)
    q = nearest_e4m3(y / torch.ldexp(torch.ones_like(m), e)[:, :, None])
    return q.view(T, -1)[:, :Hd], e


@pytest.mark.parametrize("T,Hd,x_dtype,r_dtype,w_dtype", [(65536, 2048, BF, BF, BF), (16384, 4096, BF, F32, F32),
                                                          (3000, 8208, F32, None, F32), (150, 16384, BF, F32, BF),
                                                          (20000, 1040, BF, None, F32)])
def test_8_bit_norm_is_the_definition_but_for_one_in_ten_million(cuda_device, T, Hd, x_dtype, r_dtype, w_dtype):
    g = torch.Generator(device=cuda_device).manual_seed(T + Hd)
    x = torch.randn(T, Hd, generator=g, device=cuda_device)
    x[:, ::257] *= 20
    x = x.to(x_dtype)
    r = None if r_dtype is None else (2 * torch.randn(T, Hd, generator=g, device=cuda_device)).to(r_dtype)
    w = (1 + 0.1 * torch.randn(Hd, generator=g, device=cuda_device)).to(w_dtype)
    _, h, _, q, qs = flce.flce_add_rms_norm(x, w, residual=r, eps=1e-6, normed=False, fp8=True)
    off = scales = 0
    for rows in torch.arange(T, device=cuda_device).split(4096):
        want, e = definition(h[rows], w, 1e-6)
        off += int((q[rows].double() != want).sum())
        scales += int((qs.view(torch.uint8)[rows].int() - 127 != e).sum())
    assert scales == 0
    assert off <= max(4, 8e-8 * T * Hd)


@pytest.mark.parametrize("lengths", [[5000, 4000], [300, 200] * 16, [60000, 45000], [1500, 700, 4097, 1] * 40])
@pytest.mark.parametrize("length_normalize", [False, True])
def test_rewards_are_rounded_once(cuda_device, lengths, length_normalize):
    """Log ratios of both signs that cancel in the sum, which plain fp32 sums would miss by 100 times the bound."""
    T = sum(lengths)
    g = torch.Generator(device=cuda_device).manual_seed(T)
    logp = -6 * torch.rand(T, generator=g, device=cuda_device)
    ref = logp + 3 * torch.randn(T, generator=g, device=cuda_device)
    y = torch.ones(T, dtype=torch.int64, device=cuda_device)
    y[torch.rand(T, generator=g, device=cuda_device) < 0.2] = IGN
    cu = cu_of(lengths, cuda_device)
    _, _, chosen, rejected, ws = flce.flce_preference_loss(logp, y, cu, ref_logp=ref, beta=0.25,
                                                           length_normalize=length_normalize)
    assert flce.flce_read_device_status(ws) == 0
    at = y != IGN
    seq = torch.searchsorted(cu, torch.arange(T, device=cuda_device), right=True)[at] - 1
    d = (logp - ref)[at].double()
    zero = torch.zeros(len(lengths), dtype=torch.float64, device=cuda_device)
    n = zero.index_add(0, seq, torch.ones_like(d)).clamp(min=1) if length_normalize else 1.0
    want = 0.25 * zero.index_add(0, seq, d) / n
    size = 0.25 * zero.index_add(0, seq, d.abs()) / n
    got = torch.stack([chosen, rejected], 1).reshape(-1).double()
    assert bool(((got - want).abs() <= 2.0 ** -24 * want.abs() * (1 + 1e-6) + 2.0 ** -40 * size).all())
