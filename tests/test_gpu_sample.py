"""Drawing tokens against the definition in 64 bits, row by row.

The kernel's weights are good to 2^-31 and their sums exact, the oracle's sums to 2^-52 a step: on inputs drawn at
random the two fall on different sides of a border with a chance of one in a million for a row of 250,000
equally likely words and far less for others, so tokens have to be equal.  logp is a logarithm of a ratio good to 2^-31 and
rounded to fp32: half a step of the result, one of log(mantissa) in [0, log 2), and 2^-31 of the weight.
"""

import math

import numpy as np
import pytest
import torch

import lm_head_linear_gb300 as flce
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

BF, F32, I64 = torch.bfloat16, torch.float32, torch.int64
IGN = -100


def draw_row(l, u, temp, k, p, mp):
    """One row from the definition; l in 64 bits."""
    l = np.where(np.isnan(l), -np.inf, l)
    ids = np.flatnonzero(l > -np.inf)
    if ids.size == 0:
        return IGN, 0.0
    best = l.max()
    if not temp > 0:
        return int(np.flatnonzero(l == best)[0]), 0.0
    if best == np.inf:
        ids = np.flatnonzero(l == np.inf)
        w = np.ones(ids.size)
    else:
        ids = ids[np.argsort(-l[ids], kind="stable")]
        w = np.exp((l[ids] - best) / temp)
    if k > 0:
        ids, w = ids[:k], w[:k]
    if p < 1:
        c = np.cumsum(w)
        keep = (c - w) < p * c[-1]
        keep[0] = True
        ids, w = ids[keep], w[keep]
    if mp > 0:
        ids, w = ids[w >= min(mp, 1.0)], w[w >= min(mp, 1.0)]
    order = np.argsort(ids, kind="stable")
    ids, w = ids[order], w[order]
    c = np.cumsum(w)
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    i = int(np.searchsorted(c, u * c[-1], side="right"))
    return int(ids[i]), float(np.log(w[i] / c[-1]))


def check(logits, u, temp=1.0, k=0, p=1.0, mp=0.0, **kw):
    T = logits.shape[0]
    tokens, logp = flce.flce_sample(logits, u, temperature=temp, top_k=k, top_p=p, min_p=mp, **kw)
    assert tokens.dtype == I64 and logp.dtype == F32 and tokens.shape == logp.shape == (T,)
    rows, us = logits.double().cpu().numpy(), u.double().cpu().numpy()
    per = [v.double().cpu().tolist() if torch.is_tensor(v) else [v] * T for v in (temp, k, p, mp)]
    want = [draw_row(rows[r], us[r], per[0][r], int(per[1][r]), per[2][r], per[3][r]) for r in range(T)]
    got, lp = tokens.cpu().tolist(), logp.double().cpu().tolist()
    assert got == [w[0] for w in want], [(r, a, b[0]) for r, (a, b) in enumerate(zip(got, want)) if a != b[0]][:5]
    for a, (_, b) in zip(lp, want):
        assert abs(a - b) <= 2.0 ** -24 * abs(b) + 2.0 ** -24 + 2.0 ** -29, (a, b)


def rows_of(T, V, dev, dtype=BF, seed=0, spread=2.0, peaks=20, pad=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    l = torch.randn(T, V + pad, generator=g, device=dev) * spread
    if peaks:
        l.scatter_add_(1, torch.randint(0, V, (T, peaks), generator=g, device=dev),
                       14 * torch.rand(T, peaks, generator=g, device=dev))
    return l.to(dtype)[:, :V], torch.rand(T, generator=g, device=dev)


SIZES = [(1, 1), (3, 2), (5, 7), (2, 8), (4, 33), (9, 1000), (3, 4097), (1, 32000), (40, 32001), (2, 124160), (5, 100003), (1, 248320),
         (2, 248321), (700, 300)]
SETTINGS = [dict(), dict(temp=0.7), dict(temp=0.0), dict(k=1), dict(k=50), dict(p=0.9), dict(mp=0.05), dict(k=50, p=0.95, mp=0.02, temp=0.8),
            dict(k=900, p=0.999), dict(temp=1.7, p=0.98), dict(k=5000), dict(k=5000, p=0.99, temp=3.0), dict(p=1e-6), dict(p=0.0),
            dict(mp=1.0), dict(k=1 << 40), dict(temp=30.0, p=0.5), dict(temp=30.0, mp=0.9), dict(temp=1e-4), dict(temp=1e300, p=0.7)]


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_settings(cuda_device, T, V, dtype):
    for i, s in enumerate(SETTINGS):
        l, u = rows_of(T, V, cuda_device, dtype, seed=T * V + i)
        check(l, u, **s)


@pytest.mark.parametrize("V", [4097, 124160, 393216])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.3, 1.0])
def test_flat_rows(cuda_device, V, dtype, spread):
    """Prefixes of hundreds of thousands of words, with many equals: more than the sorted list holds."""
    for i, s in enumerate([dict(), dict(p=0.5), dict(p=0.95), dict(k=V // 2), dict(k=V // 3, p=0.9), dict(mp=0.3), dict(k=V // 2, p=0.3, mp=0.2),
                           dict(k=V), dict(k=V - 1, p=0.9999)]):
        l, u = rows_of(2, V, cuda_device, dtype, seed=V + i, spread=spread, peaks=0)
        if spread == 0.0 and "p" in s:  # exact ties at p's border: p V a whole number, in the oracle's sums as well
            s = dict(s, p=0.5)
        check(l, u, **s)


def test_equal_words_exactly(cuda_device):
    """1024 equal words: u = i / 1024 draws word i, the number before it word i - 1; filters keep the lowest indexes."""
    i = torch.arange(1024, device=cuda_device)
    l = torch.full((1024, 1024), -3.25, device=cuda_device)
    tokens, logp = flce.flce_sample(l, i / 1024)
    assert torch.equal(tokens, i) and bool(((logp + math.log(1024)).abs() < 1e-6).all())
    before = torch.nextafter(i / 1024, torch.zeros(1024, device=cuda_device))
    assert torch.equal(flce.flce_sample(l, before)[0], (i - 1).clamp(min=0))
    assert torch.equal(flce.flce_sample(l, i / 1024, top_k=256)[0], i // 4)
    assert torch.equal(flce.flce_sample(l, i / 1024, top_p=0.5)[0], i // 2)
    assert torch.equal(flce.flce_sample(l, i / 1024, top_k=512, top_p=0.5)[0], i // 4)
    assert torch.equal(flce.flce_sample(l, i / 1024, temperature=0.0)[0], torch.zeros_like(i))
    assert torch.equal(flce.flce_sample(l, i / 1024, min_p=1.0)[0], i)
    l[:, 7] = 4.0  # 1024 - 1 equals behind one
    assert torch.equal(flce.flce_sample(l, i / 1024, top_k=1)[0], torch.full_like(i, 7))
    assert torch.equal(flce.flce_sample(l, torch.full_like(l[0], 0.999999), top_k=4, temperature=1e6)[0], torch.full_like(i, 7))
    assert torch.equal(flce.flce_sample(l, torch.zeros_like(l[0]), top_k=4, temperature=1e6)[0], torch.zeros_like(i))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks_infinities_and_nan(cuda_device, dtype):
    T, V = 12, 5003
    l, u = rows_of(T, V, cuda_device, dtype, seed=5)
    l = l.contiguous()
    inf, nan = float("inf"), float("nan")
    l[0] = -inf
    l[1] = nan
    l[2] = -inf
    l[2, 4321] = -1e30
    l[3, ::2] = nan
    l[4, 3:] = -inf
    l[5, 77], l[5, 4000], l[5, 4001] = inf, inf, inf
    l[6] = torch.finfo(dtype).min
    l[7, :5000] = torch.finfo(dtype).min
    l[8] = torch.finfo(dtype).max
    l[9, 10], l[9, 11] = torch.finfo(dtype).max, torch.finfo(dtype).min
    l[10, ::2] = 0.0
    l[10, 1::2] = -0.0
    l[11, 0], l[11, 1] = inf, nan
    for s in (dict(), dict(k=3), dict(p=0.7), dict(mp=0.1), dict(k=4000, p=0.9), dict(temp=0.0), dict(temp=1e300), dict(temp=0.01, p=0.6)):
        check(l, u, **s)
    tokens, logp = flce.flce_sample(l, u, ignore_index=-1)
    assert tokens[0] == -1 and tokens[1] == -1 and logp[0] == 0 and tokens[2] == 4321


@pytest.mark.parametrize("V", [4097, 40000, 250000])
@pytest.mark.parametrize("octaves", [44.2, 45.1, 46.5, 47.9, 60.0])
def test_words_without_a_weight(cuda_device, V, octaves):
    """Few words with a weight and thousands just below the least one."""
    l = torch.full((4, V), -octaves * math.log(2.0), device=cuda_device)
    l[:, 17] = 0.0
    l[1, 1000:1400] = -1.0
    l[2, ::5] = -octaves * math.log(2.0) + 0.01
    l[3, 1::3] = float("-inf")
    u = torch.tensor([0.3, 0.9, 0.5, 0.999], device=cuda_device)
    for s in (dict(p=0.995), dict(k=2000, p=0.995), dict(k=700, p=0.999), dict(k=2000), dict(k=30), dict(p=0.5)):
        check(l, u, **s)
        check(l * 0.3, u, temp=0.3, **s)


def test_logp_of_words_that_are_nearly_certain(cuda_device):
    """One word far ahead: its logp is the others' weight to 2^-21 of itself (sums good to 2^-29, fp32 logarithm) and
    half a unit of 2^-46 for each of the 199 others (over this one's weight, at least 2^(-1/32)); 0 where it is alone."""
    gaps = torch.tensor([2.0, 5.0, 9.0, 14.0, 18.0], dtype=F32, device=cuda_device)
    l = torch.zeros(5, 3000, device=cuda_device)
    l[:, 100:200] = torch.linspace(-1, 0, 100, device=cuda_device)
    l[:, 200:] = float("-inf")
    l[:, 7] = gaps + 3
    tokens, logp = flce.flce_sample(l, torch.full((5,), 0.5, device=cuda_device), temperature=0.7)
    assert torch.equal(tokens[1:], torch.full_like(tokens[1:], 7))
    z = l.double() / 0.7
    others = torch.where(torch.arange(3000, device=cuda_device) == 7, -math.inf, z)
    want = -torch.log1p(torch.exp(torch.logsumexp(others, 1) - z[:, 7]))
    assert bool(((logp.double() - want).abs() <= 2.0 ** -21 * want.abs() + 199 * 2.0 ** -47 * 1.03)[1:].all())
    _, alone = flce.flce_sample(l, torch.full((5,), 0.5, device=cuda_device), top_k=2, top_p=0.5)
    assert bool((alone[1:] == 0).all())
    for s in (dict(top_k=1), dict(top_p=1e-9), dict(min_p=1.0)):
        assert bool((flce.flce_sample(l, torch.full((5,), 0.9, device=cuda_device), **s)[1] == 0).all())


def test_random_numbers_out_of_range(cuda_device):
    l, _ = rows_of(8, 1000, cuda_device, F32, seed=3)
    l = l[:1].expand(8, 1000).contiguous()
    u = torch.tensor([-1.0, float("nan"), -0.0, 0.0, 1.0, 2.0, float("inf"), 1 - 2.0 ** -24], device=cuda_device)
    check(l, u)
    check(l, u, k=20)
    t = flce.flce_sample(l, u)[0]
    assert bool((t[:4] == t[0]).all()) and bool((t[4:] == t[7]).all())


def test_settings_of_each_row(cuda_device):
    T, V = 300, 9001
    g = torch.Generator(device=cuda_device).manual_seed(1)
    r = lambda: torch.rand(T, generator=g, device=cuda_device)
    l, u = rows_of(T, V, cuda_device, BF, seed=8, pad=3)
    temp = torch.where(r() < 0.2, 0.0, 0.2 + 2 * r())
    k = torch.where(r() < 0.3, 0, torch.randint(1, 3000, (T,), generator=g, device=cuda_device)).int()
    p = torch.where(r() < 0.3, 1.0, r())
    mp = torch.where(r() < 0.3, 0.0, 0.3 * r())
    check(l, u, temp, k, p, mp)
    temp[:4] = torch.tensor([-1.0, float("nan"), float("inf"), 1.0], device=cuda_device)
    k[:4] = torch.tensor([0, 0, 0, -5], device=cuda_device)
    p[2:4], mp[2:4] = torch.tensor([1.0, 1.5], device=cuda_device), torch.tensor([0.0, -2.0], device=cuda_device)
    check(l, u, temp, k, p, mp)
    check(l, u, 0.9, k, 0.95, mp)


@pytest.mark.parametrize("V", [12345, 32001, 248320, 393216])
@pytest.mark.parametrize("shift", [-40.0, -3.0, -0.25, 0.0, 0.25, 3.0, 40.0])
def test_nuclei_of_rows_with_few_values(cuda_device, V, shift):
    """bf16 rows have some thousand values: nuclei that end at positive ones, at negative ones, close to 0 (where values
    have no end) and with min-p, and rows with masks, infinities, or more values than are counted."""
    for i, s in enumerate([dict(p=0.5), dict(p=0.95), dict(p=0.9999, mp=1e-4), dict(p=0.99, temp=4.0, mp=0.01), dict(p=0.1, temp=0.3),
                           dict(p=0.9, temp=100.0)]):
        for spread in (0.02, 2.0):
            l, u = rows_of(4, V, cuda_device, BF, seed=V + i, spread=spread, peaks=0)
            l = (l.float() + shift).to(BF)
            l[1, ::3] = float("-inf")
            l[2, 1::2] = float("nan")
            l[3, 1:4000] *= 2.0 ** -12  # many close to 0
            check(l, u, **s)


@pytest.mark.parametrize("V", [12345, 32001, 248320])
@pytest.mark.parametrize("shift", [-40.0, -0.25, 0.0, 3.0])
def test_top_k_of_rows_with_few_values(cuda_device, V, shift):
    """The k-th logit among many equals, at positive values, negative ones and close to 0, alone and before top-p and min-p;
    k above the number of words that are not masked."""
    for i, s in enumerate([dict(k=100), dict(k=300), dict(k=700, p=0.9), dict(k=1000, p=0.99, mp=0.01), dict(k=3000), dict(k=V // 2, p=0.7),
                           dict(k=V // 2 + 1, temp=9.0), dict(k=V - 1), dict(k=V - 1, p=0.99999)]):
        for spread in (0.02, 2.0):
            l, u = rows_of(4, V, cuda_device, BF, seed=V + i, spread=spread, peaks=0)
            l = (l.float() + shift).to(BF)
            l[1, ::3] = float("-inf")
            l[2, 1::2] = float("nan")
            l[3, 1:4000] *= 2.0 ** -12
            check(l, u, **s)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinite_temperature(cuda_device, dtype):
    """Every word that is not masked weighs 1, whatever its logit and whatever min_p up to 1."""
    l, _ = rows_of(16, 4097, cuda_device, dtype, seed=41)
    l = l.clone()
    l[3, ::2] = float("-inf")
    u = (torch.arange(16, device=cuda_device) + 0.5) / 16
    temp = torch.full((16,), float("inf"), device=cuda_device)
    for mp in (0.0, 0.5, 1.0, torch.linspace(0, 1, 16, device=cuda_device)):
        check(l, u, temp=temp, mp=mp)
        check(l, u, temp=temp, mp=mp, k=1000)
    _, logp = flce.flce_sample(l, u, temperature=temp, min_p=1.0)
    assert abs(logp[0].item() + math.log(4097)) <= 1e-6



@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,pad,offset", [(33, 1, 1), (1000, 3, 5), (4097, 0, 3), (4096, 7, 0), (50257, 2, 7), (13, 0, 2)])
def test_rows_of_any_alignment_and_guards(cuda_device, dtype, V, pad, offset):
    """Rows that start anywhere and lie V + pad apart; what is between them (NaN) counts for nothing; nothing but the
    outputs is written."""
    T = 17
    buf = torch.full((T * (V + pad) + 64,), float("nan"), dtype=dtype, device=cuda_device)
    l = torch.as_strided(buf, (T, V), (V + pad, 1), 16 + offset)
    src, u = rows_of(T, V, cuda_device, dtype, seed=V)
    l.copy_(src)
    kept = buf.clone()
    tok, lp = Guarded((T,), I64, cuda_device), Guarded((T,), F32, cuda_device)
    for s in (dict(), dict(k=9, p=0.9), dict(p=0.8)):
        check(l, u, **s, out={"tokens": tok.t, "logp": lp.t})
        assert tok.intact() and lp.intact()
    assert torch.equal(torch.nan_to_num(buf, 3.0), torch.nan_to_num(kept, 3.0))


def test_many_rows_offsets_past_32_bits_and_streams(cuda_device):
    l = torch.zeros(20000, 120000, dtype=BF, device=cuda_device)  # 2.4e9 logits
    l[:, 5] = 1.0
    l[-1, 119999] = 40.0
    u = torch.rand(20000, device=cuda_device)
    tokens, _ = flce.flce_sample(l, u, top_k=2)
    first = torch.exp(torch.tensor(-1.0, dtype=torch.float64)) / (1 + torch.exp(torch.tensor(-1.0, dtype=torch.float64)))
    assert torch.equal(tokens[:-1], torch.where(u[:-1].double() < float(first), 0, 5)) and tokens[-1] == 119999
    del l
    a, ua = rows_of(64, 32000, cuda_device, BF, seed=1)
    b, ub = rows_of(3, 200000, cuda_device, F32, seed=2)
    want = flce.flce_sample(a, ua, top_p=0.9), flce.flce_sample(b, ub, top_k=2000)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        x = flce.flce_sample(a, ua, top_p=0.9, stream=s1)
        y = flce.flce_sample(b, ub, top_k=2000, stream=s2)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(x + y, want[0] + want[1]))


def test_captured_call(cuda_device):
    l, u = rows_of(5, 70001, cuda_device, BF, seed=4)
    l = l.contiguous()
    out = {"tokens": torch.empty(5, dtype=I64, device=cuda_device), "logp": torch.empty(5, device=cuda_device)}
    flce.flce_sample(l, u, top_k=40, top_p=0.9, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        flce.flce_sample(l, u, top_k=40, top_p=0.9, out=out)
    for seed in (11, 12):
        l2, u2 = rows_of(5, 70001, cuda_device, BF, seed=seed)
        l.copy_(l2), u.copy_(u2)
        want = [x.clone() for x in flce.flce_sample(l, u, top_k=40, top_p=0.9)]
        g.replay()
        assert torch.equal(out["tokens"], want[0]) and torch.equal(out["logp"], want[1])
        check(l, u, k=40, p=0.9)


def test_frequencies(cuda_device):
    """200,000 draws from one row of 50 words: each word's share is its probability (5 standard deviations)."""
    T = 200000
    g = torch.Generator(device=cuda_device).manual_seed(9)
    row = torch.randn(50, generator=g, device=cuda_device)
    tokens, logp = flce.flce_sample(row.expand(T, 50).contiguous(), torch.rand(T, generator=g, device=cuda_device), temperature=0.8)
    p = torch.softmax(row.double() / 0.8, 0)
    share = torch.bincount(tokens, minlength=50).double() / T
    assert bool(((share - p).abs() <= 5 * (p * (1 - p) / T).sqrt() + 1.0 / T).all())
    assert bool(((logp.double() - p.log()[tokens]).abs() < 1e-6).all())


def test_refusals(cuda_device):
    l, u = rows_of(4, 100, cuda_device)
    f = flce.flce_sample
    for kw in (dict(temperature=torch.ones(3, device=cuda_device)), dict(top_k=torch.ones(4, device=cuda_device)),
               dict(top_k=torch.ones(4, device=cuda_device, dtype=I64)), dict(top_p=torch.ones(4)), dict(min_p=torch.ones(4, 1, device=cuda_device)),
               dict(out={"tokens": torch.empty(4, device=cuda_device)})):
        with pytest.raises(ValueError):
            f(l, u, **kw)
    with pytest.raises(ValueError):
        f(l, u[:3])
    with pytest.raises(ValueError):
        f(l.half(), u)
    with pytest.raises(ValueError):
        f(l.t(), torch.rand(100, device=cuda_device))
    with pytest.raises(TypeError):
        f(l, u, temperature="warm")
    nan = float("nan")
    for kw in (dict(temperature=-1.0), dict(temperature=nan), dict(top_p=-0.1), dict(top_p=1.1), dict(top_p=nan), dict(min_p=-0.1),
               dict(min_p=1.5), dict(min_p=nan), dict(ignore_index=5)):
        with pytest.raises(flce.FlceError) as e:
            f(l, u, **kw)
        assert e.value.status == 1
    with pytest.raises(flce.FlceError) as e:
        f(torch.zeros(1, 393217, device=cuda_device), u[:1])
    assert e.value.status == 2
    with pytest.raises(flce.FlceError) as e:
        f(l[:1].expand(4, 100), u)  # rows on top of one another
    assert e.value.status == 1
    t, lp = f(torch.empty(0, 100, device=cuda_device), torch.empty(0, device=cuda_device))
    assert t.shape == (0,) and lp.shape == (0,)
