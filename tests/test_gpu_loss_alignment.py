"""The losses on arrays off 16 bytes: each per-token array in turn starts one element into a buffer.  The same
bits as with aligned arrays, and nothing written around the outputs."""

import pytest
import torch

import lm_head_linear_gb300 as flce

from test_gpu_losses import cu_of, draw

pytestmark = pytest.mark.gpu


def shifted(t):
    """A copy of `t` one element into a buffer (off 16 bytes), and that buffer."""
    buf = torch.full((t.numel() + 9,), 77, dtype=t.dtype, device=t.device)
    v = buf[1:1 + t.numel()]
    v.copy_(t)
    assert v.data_ptr() % 16 and v.is_contiguous()
    return v, buf


def around(buf, n):
    return bool((buf[:1] == 77).all()) and bool((buf[1 + n:] == 77).all())


INPUTS = ("logp", "old", "adv", "y", "ref", "dloss")


@pytest.mark.parametrize("T", [3, 5003, 40003])
@pytest.mark.parametrize("reduction", ["none", "mean", "sequence_mean"])
@pytest.mark.parametrize("which", INPUTS + ("dlogp", "loss", "all"))
def test_policy(cuda_device, T, reduction, which):
    logp, old, ref, adv, y, g = draw(T, cuda_device, seed=T)
    cu = cu_of([T // 3, 0, T - T // 3 - 1], cuda_device, start=1)
    n = T if reduction == "none" else 1
    a = {"logp": logp, "old": old, "adv": adv, "y": y, "ref": ref,
         "dloss": torch.randn(n, generator=g, device=cuda_device)}
    out = {"dlogp": torch.empty(T, device=cuda_device), "loss": torch.empty(n, device=cuda_device)}

    def call():
        r = flce.flce_policy_loss(a["logp"], a["old"], a["adv"], a["y"], ref_logp=a["ref"], cu_seqlens=cu, reduction=reduction,
                                  dloss=a["dloss"], kl_coef=0.1, out=dict(out))
        assert flce.flce_read_device_status(r[-1]) == 0
        return [t.clone() for t in r[:4]]

    want = call()
    bufs = []
    for k in INPUTS + ("dlogp", "loss") if which == "all" else (which,):
        d = a if k in a else out
        d[k], buf = shifted(d[k])
        bufs.append((buf, d[k].numel()))
    assert all(torch.equal(x, z) for x, z in zip(want, call()))
    assert all(around(b, n) for b, n in bufs)


@pytest.mark.parametrize("lengths", [[1, 2], [700, 333, 64, 9], [9000, 8001], [5, 0, 41, 50] * 30])
@pytest.mark.parametrize("which", ["logp", "ref", "y", "dlogp", "all"])
def test_preference(cuda_device, lengths, which):
    T = sum(lengths) + 5
    logp, _, ref, _, y, _ = draw(T, cuda_device, seed=T)
    cu = cu_of(lengths, cuda_device, start=3)
    a, out = {"logp": logp, "ref": ref, "y": y}, {"dlogp": torch.empty(T, device=cuda_device)}

    def call():
        r = flce.flce_preference_loss(a["logp"], a["y"], cu, ref_logp=a["ref"], out=dict(out))
        assert flce.flce_read_device_status(r[-1]) == 0
        return [t.clone() for t in r[:4]]

    want = call()
    bufs = []
    for k in ("logp", "ref", "y", "dlogp") if which == "all" else (which,):
        d = a if k in a else out
        d[k], buf = shifted(d[k])
        bufs.append((buf, d[k].numel()))
    assert all(torch.equal(x, z) for x, z in zip(want, call()))
    assert all(around(b, n) for b, n in bufs)
