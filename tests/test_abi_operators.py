"""Argument checks of the operators around the head that need no device: bad sizes, NULLs,
alignment and workspaces are refused before anything is launched."""

import ctypes

import pytest

import lm_head_linear_gb300 as flce
from lm_head_linear_gb300 import build as flce_build

P = ctypes.c_void_p
OK = 4096


@pytest.fixture(scope="module")
def lib():
    flce_build.build()
    return flce.load_library()


def call(f, defaults, **kw):
    a = {**defaults, **kw}
    assert set(a) == set(defaults)
    return f(*(P(v) if isinstance(v, int) and k.isupper() and k not in SIZES else v for k, v in a.items()))


# upper-case names are pointers, but for these
SIZES = {"T", "K", "V", "S"}
NORM = dict(X=OK, x_dtype=0, ldx=128, R=OK, r_dtype=0, ldr=128, W=OK, w_dtype=0, T=4, Hd=128, eps=1e-6, H=OK, ldh=128, Y=OK,
            RSTD=OK, Q=OK, QS=OK, STREAM=None)
NORM_B = dict(DY=OK, dy_dtype=0, lddy=128, H=OK, h_dtype=0, ldh=128, W=OK, w_dtype=0, RSTD=OK, DH=None, lddh=0, T=4, Hd=128,
              DX=OK, DW=OK, WS=OK, bytes=1 << 20, STREAM=None)
QUANT = dict(A=OK, dtype=0, lda=128, rows=4, K=128, block=128, Q=OK, QS=OK, STREAM=None)
LIN = dict(X=OK, XS=OK, W=OK, WS_=OK, T=4, K=128, V=100, Y=OK, y_dtype=0, ldy=100, WS=OK, bytes=256, STREAM=None)
POL = dict(DLOSS=None, LOGP=OK, OLD=OK, REF=OK, ADV=OK, per=0, Y=OK, CU=OK, S=2, T=4, ign=-100, red=1, lo=0.2, hi=0.2, dual=0.0,
           klc=0.1, kl=3, LOSS=OK, DLOGP=OK, STATS=OK, NV=OK, WS=OK, bytes=1 << 20, STREAM=None)
PREF = dict(DLOSS=None, LOGP=OK, REF=OK, Y=OK, CU=OK, P_=2, T=4, ign=-100, red=1, kind=0, beta=0.1, smooth=0.0, margin=0.0, norm=0,
            LOSS=OK, DLOGP=OK, C=OK, R=OK, WS=OK, bytes=1 << 20, STREAM=None)
PREF = {("pairs" if k == "P_" else k): v for k, v in PREF.items()}

CASES = [
    ("flce_add_rms_norm", NORM, [
        (1, dict(T=-1)), (1, dict(T=1 << 30)), (1, dict(Hd=0)), (2, dict(Hd=120)), (2, dict(Hd=16400)), (1, dict(x_dtype=2)),
        (1, dict(r_dtype=-1)), (1, dict(w_dtype=7)), (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))), (1, dict(X=None)),
        (1, dict(W=None)), (1, dict(H=None)), (1, dict(R=None)), (1, dict(QS=None)), (1, dict(Y=None, Q=None, QS=None)),
        (3, dict(ldx=120)), (3, dict(ldx=129)), (3, dict(ldr=132)), (3, dict(ldh=64)), (3, dict(X=OK + 8)), (3, dict(Q=OK + 8)),
        (3, dict(RSTD=OK + 2))]),
    ("flce_add_rms_norm_backward", NORM_B, [
        (1, dict(T=-1)), (2, dict(Hd=24)), (1, dict(dy_dtype=3)), (1, dict(DY=None)), (1, dict(DW=None)), (1, dict(RSTD=None)),
        (3, dict(ldh=130)), (3, dict(DH=OK, lddh=100)), (3, dict(DX=OK + 4)), (3, dict(DW=OK + 1)), (4, dict(WS=None)),
        (4, dict(bytes=100)), (3, dict(WS=OK + 16))]),
    ("flce_quantize_fp8", QUANT, [
        (1, dict(rows=-1)), (1, dict(K=0)), (2, dict(K=40, lda=40)), (1, dict(dtype=2)), (1, dict(block=64)), (1, dict(A=None)),
        (1, dict(QS=None)), (3, dict(lda=130)), (3, dict(A=OK + 2))]),
    ("flce_linear_fp8", LIN, [
        (1, dict(T=-1)), (1, dict(V=0)), (1, dict(K=0)), (1, dict(K=1 << 24)), (2, dict(K=24)), (1, dict(y_dtype=2)), (1, dict(X=None)),
        (1, dict(WS_=None)), (1, dict(Y=None)), (1, dict(ldy=99)), (3, dict(X=OK + 8)), (3, dict(W=OK + 1)), (3, dict(Y=OK + 1)),
        (4, dict(WS=None)), (4, dict(bytes=255)), (3, dict(WS=OK + 128))]),
    ("flce_policy_loss", POL, [
        (1, dict(T=-1)), (1, dict(S=-1)), (1, dict(red=4)), (1, dict(red=-1)), (1, dict(kl=0)), (1, dict(kl=4)), (1, dict(lo=1.0)),
        (1, dict(lo=-0.1)), (1, dict(hi=-0.1)), (1, dict(hi=float("nan"))), (1, dict(dual=1.0)), (1, dict(dual=-2.0)),
        (1, dict(klc=float("inf"))), (1, dict(REF=None)), (1, dict(CU=None, red=3)), (1, dict(CU=None, per=1)),
        (1, dict(LOSS=None, DLOGP=None)), (1, dict(LOGP=None)), (1, dict(Y=None)), (1, dict(ADV=None)), (3, dict(LOGP=OK + 2)),
        (3, dict(Y=OK + 4)), (3, dict(CU=OK + 4)), (3, dict(NV=OK + 4)), (4, dict(WS=None)), (4, dict(bytes=256)),
        (3, dict(WS=OK + 64))]),
    ("flce_preference_loss", PREF, [
        (1, dict(T=-1)), (1, dict(pairs=-1)), (1, dict(red=3)), (1, dict(kind=3)), (1, dict(beta=0.0)), (1, dict(beta=-1.0)),
        (1, dict(beta=float("inf"))), (1, dict(smooth=0.5)), (1, dict(smooth=0.1, kind=1)), (1, dict(margin=0.1, kind=2)),
        (1, dict(margin=float("nan"))), (1, dict(LOSS=None, DLOGP=None)), (1, dict(CU=None)), (1, dict(LOGP=None)),
        (3, dict(LOGP=OK + 1)), (3, dict(CU=OK + 4)), (4, dict(WS=None)), (4, dict(bytes=256)), (3, dict(WS=OK + 8))]),
]


@pytest.mark.parametrize("name,defaults,status,change",
                         [(n, d, st, ch) for n, d, cases in CASES for st, ch in cases])
def test_refused_on_the_host(lib, name, defaults, status, change):
    assert call(getattr(lib, name), defaults, **change) == status
    assert len(lib.flce_last_error()) > 0


def test_workspace_sizes(lib):
    assert lib.flce_linear_fp8_workspace_size(0, 128, 5) == 256 and lib.flce_linear_fp8_workspace_size(-1, 128, 5) == 0
    assert lib.flce_policy_loss_workspace_size(-1, 0) == 0 and lib.flce_policy_loss_workspace_size(10, -1) == 0
    assert lib.flce_preference_loss_workspace_size(-1) == 0
    assert lib.flce_add_rms_norm_backward_workspace_size(10, 0) == 0
    last = 0
    for T in (0, 1, 1000, 32768, 131072, 1 << 20, 1 << 25):  # grows with T, by about a third of a byte per token
        now = lib.flce_policy_loss_workspace_size(T, 10)
        assert last <= now <= 200_000 + T // 3
        last = now
    assert lib.flce_preference_loss_workspace_size(1000) >= 12 * 1000
    assert lib.flce_status_string(8) == b"FLCE_ERR_SEQUENCES"


def test_the_operators_refuse_tensors_of_the_host():
    import torch
    x, w = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(32)
    v, y = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    for f in (lambda: flce.flce_add_rms_norm(x, w), lambda: flce.flce_add_rms_norm_backward(x, x, w, v),
              lambda: flce.flce_quantize_fp8(x), lambda: flce.flce_policy_loss(v, v, v, y),
              lambda: flce.flce_preference_loss(v, y, y), lambda: flce.flce_linear_fp8(x, w, x, w),
              lambda: flce.flce_add_rms_norm(None, w), lambda: flce.flce_add_rms_norm(x, 3)):
        with pytest.raises(ValueError):
            f()
