"""Drawing tokens from fp32 rows whose logits over the temperature lie far from 0 (up to some thousand octaves).

The product of a logit and log2(e) / temperature is then rounded to up to 2^-12, so counting by steps of 1/32 octave may
file a word under a step that its weight has left by that much.  Prefixes longer than the sorted list end by such counts.

Every border is put in the middle of a word: a prefix of m words ends half way through its last one, a random number lies
half way through the drawn word's share.  The oracle's weights are exact to 2^-50, the kernel's to 2^-28, half a word of at most
60,000 similar ones is 2^-17 of the sum: tokens have to be equal.  logp as in test_gpu_sample.py.
"""

import math

import numpy as np
import pytest
import torch

import lm_head_linear_gb300 as flce

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def check_prefixes(row, temp, k, lengths, dev, mp=0.0):
    """row: one row of logits (fp32 numpy).  top-k k (0: all), then top-p with prefixes of `lengths` words."""
    l = row.astype(np.float64)
    order = np.argsort(-l, kind="stable")
    w = np.exp((l[order] - l[order[0]]) / temp)
    n = min(k, l.size) if k else l.size
    c = np.cumsum(w[:n])
    logits = torch.from_numpy(row).to(dev)
    for m in lengths:
        p = float((c[m - 1] - 0.5 * w[m - 1]) / c[-1])
        keep = order[:m][w[:m] >= mp]
        ids = np.sort(keep)
        wi = np.exp((l[ids] - l[order[0]]) / temp)
        ci = np.cumsum(wi)
        last, lightest = int(np.flatnonzero(ids == keep[-1])[0]), int(np.argmin(wi))
        at = sorted({0, last, lightest, ids.size // 3, ids.size - 1})  # places of the drawn words
        u = torch.tensor([(ci[i] - 0.5 * wi[i]) / ci[-1] for i in at], dtype=torch.float32, device=dev)
        tokens, logp = flce.flce_sample(logits.expand(len(at), -1).contiguous(), u, temperature=temp, top_k=k, top_p=p, min_p=mp)
        assert tokens.tolist() == [int(ids[i]) for i in at], (m, p, at)
        want = np.log(wi[at] / ci[-1])
        assert (np.abs(logp.double().cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -24 + 2.0 ** -28).all()


def beside_a_step(top, width, temp, side):
    """The fp32 logit within `width` below `top` whose exact product lies furthest above (side 1) or below (-1) the
    middle of the step that the rounded product falls into, seen from the row's largest."""
    c = LOG2E / temp
    c_hi = np.float32(c)
    bits = np.float32(top).view(np.int32)
    n = 4_000_000
    l = np.arange(bits - n, bits, dtype=np.int32).view(np.float32) if top > 0 else np.arange(bits + 1, bits + n, dtype=np.int32).view(np.float32)
    l = l[l >= np.float32(top) - np.float32(width)]
    step = np.round(32 * (l * c_hi).astype(np.float64)) / 32
    off = l.astype(np.float64) * c - step
    return l[np.argmax(side * off)]


OFFSETS = [(800.0, 1.0), (1500.0, 1.0), (5000.0, 1.0), (5600.0, 1.0), (-5000.0, 1.0), (20.0, 0.004), (3.0, 0.00061)]


@pytest.mark.parametrize("top,temp", OFFSETS)
@pytest.mark.parametrize("side", [1, -1])
def test_two_values_beside_a_step(cuda_device, top, temp, side):
    """The end of the prefix within a few words of where one value's words end, top-p alone (few of the heavier value) and
    after top-k (half and half)."""
    rng = np.random.default_rng(int(abs(top)))
    heavy = beside_a_step(top, 0.9 * temp, temp, side)
    light = beside_a_step(top - 1.1 * temp, 0.9 * temp, temp, -side)
    assert light < heavy < np.float32(top)
    for count, V, k in ((400, 60000, 0), (20000, 60000, 0), (20000, 60000, 50000), (3000, 9001, 8000)):
        row = np.full(V, light, dtype=np.float32)
        at = rng.permutation(V)
        row[at[:count]] = heavy
        row[at[count]] = np.float32(top)
        lengths = {count + 1 + d for d in (-6, -3, -2, -1, 0, 1, 2, 3, 6)} | {count // 2, count + (V - count) // 2}
        check_prefixes(row, temp, k, sorted(m for m in lengths if 0 < m <= (k or V)), cuda_device)


@pytest.mark.parametrize("top,temp", OFFSETS)
@pytest.mark.parametrize("spread", [0.01, 0.3, 2.0])
def test_long_prefixes(cuda_device, top, temp, spread):
    """Prefixes of thousands to tens of thousands of words, top-p alone, after top-k and with min-p."""
    rng = np.random.default_rng(7)
    for V, k, mp in ((20001, 0, 0.0), (60000, 0, 0.02), (60000, 45000, 0.0), (30000, 2500, 0.0)):
        row = (top + temp * spread * rng.standard_normal(V)).astype(np.float32)
        n = k or V
        check_prefixes(row, temp, k, [n // 9, n // 2, n - n // 9], cuda_device, mp=mp if spread < 1 else 0.0)
