"""Argument checks, without a device, of the norm with a checkpoint, the 4-bit product, its quantiser and
the sampler: as test_abi_operators.py."""

import pytest

import lm_head_linear_gb300 as flce
from test_abi_operators import LIN, NORM, NORM_B, OK, QUANT, call, lib  # noqa: F401 (lib is a fixture)

QUANT4 = {k: v for k, v in QUANT.items() if k != "block"}

SAMPLE = dict(L=OK, dtype=0, ldl=100, U=OK, T=4, V=100, TEMP=None, temp=1.0, TOPK=None, k=0, TOPP=None, p=1.0, MINP=None, mp=0.0, ign=-100,
              TOKENS=OK, LOGP=OK, STREAM=None)
KEEP_B = {("Q" if k == "H" else "h_dtype" if k == "h_dtype" else k): v for k, v in NORM_B.items() if k != "ldh"}
KEEP_B = {k: v for name, value in KEEP_B.items() for k, v in ([(name, value), ("QS", OK)] if name == "Q" else [(name, value)])}
NAN = float("nan")

CASES = [
    ("flce_add_rms_norm_checkpoint", NORM, [
        (1, dict(T=-1)), (1, dict(T=1 << 30)), (1, dict(Hd=0)), (2, dict(Hd=120)), (2, dict(Hd=16400)), (1, dict(x_dtype=2)),
        (1, dict(r_dtype=-1)), (1, dict(w_dtype=7)), (1, dict(eps=-1.0)), (1, dict(X=None)), (1, dict(W=None)), (1, dict(H=None)),
        (1, dict(R=None)), (1, dict(QS=None)), (1, dict(Q=None)), (1, dict(Q=None, QS=None)), (1, dict(Y=None)), (1, dict(RSTD=None)),
        (3, dict(ldx=120)), (3, dict(ldr=132)), (3, dict(ldh=64)), (3, dict(X=OK + 8)), (3, dict(Q=OK + 8)), (3, dict(RSTD=OK + 2))]),
    ("flce_add_rms_norm_checkpoint_backward", KEEP_B, [
        (1, dict(T=-1)), (2, dict(Hd=24)), (1, dict(dy_dtype=3)), (1, dict(h_dtype=3)), (1, dict(DY=None)), (1, dict(Q=None)),
        (1, dict(QS=None)), (1, dict(DW=None)), (1, dict(RSTD=None)), (3, dict(Q=OK + 8)), (3, dict(lddy=130)),
        (3, dict(DH=OK, lddh=100)), (3, dict(DX=OK + 4)), (3, dict(DW=OK + 1)), (4, dict(WS=None)), (4, dict(bytes=100)),
        (3, dict(WS=OK + 16))]),
    ("flce_quantize_fp4", QUANT4, [
        (1, dict(rows=-1)), (1, dict(rows=1 << 30)), (1, dict(K=0)), (1, dict(K=1 << 24)), (2, dict(K=40, lda=40)), (1, dict(dtype=2)),
        (1, dict(A=None)), (1, dict(Q=None)), (1, dict(QS=None)), (3, dict(lda=130)), (3, dict(lda=112)), (3, dict(A=OK + 2)),
        (3, dict(Q=OK + 8))]),
    ("flce_linear_fp4", LIN, [
        (1, dict(T=-1)), (1, dict(T=1 << 30)), (1, dict(V=0)), (1, dict(V=1 << 30)), (1, dict(K=0)), (1, dict(K=1 << 24)), (2, dict(K=24)),
        (1, dict(y_dtype=2)), (1, dict(X=None)), (1, dict(XS=None)), (1, dict(W=None)), (1, dict(WS_=None)), (1, dict(Y=None)),
        (1, dict(ldy=99)), (3, dict(X=OK + 8)), (3, dict(W=OK + 1)), (3, dict(W=OK + 16)), (3, dict(WS_=OK + 2)), (3, dict(Y=OK + 1)),
        (4, dict(WS=None)), (4, dict(bytes=255)), (3, dict(WS=OK + 128))]),
    ("flce_sample", SAMPLE, [
        (1, dict(T=-1)), (1, dict(T=1 << 30)), (1, dict(V=0)), (2, dict(V=393217, ldl=400000)), (1, dict(dtype=2)), (1, dict(ldl=99)),
        (1, dict(ign=0)), (1, dict(ign=99)), (1, dict(temp=-0.1)), (1, dict(temp=NAN)), (1, dict(temp=float("inf"))), (1, dict(p=1.01)),
        (1, dict(p=-0.01)), (1, dict(p=NAN)), (1, dict(mp=1.01)), (1, dict(mp=-0.01)), (1, dict(mp=NAN)), (1, dict(L=None)),
        (1, dict(U=None)), (1, dict(TOKENS=None)), (3, dict(L=OK + 1)), (3, dict(L=OK + 2, dtype=1)), (3, dict(U=OK + 2)),
        (3, dict(TEMP=OK + 2)), (3, dict(TOPK=OK + 1)), (3, dict(TOPP=OK + 3)), (3, dict(MINP=OK + 2)), (3, dict(TOKENS=OK + 4)),
        (3, dict(LOGP=OK + 2))]),
]


@pytest.mark.parametrize("name,defaults,status,change", [(n, d, st, ch) for n, d, cases in CASES for st, ch in cases])
def test_refused_on_the_host(lib, name, defaults, status, change):  # noqa: F811
    assert call(getattr(lib, name), defaults, **change) == status
    assert len(lib.flce_last_error()) > 0


def test_workspace_sizes(lib):  # noqa: F811
    assert flce.flce_linear_fp4_workspace_size(1, 2048, 124160) >= 256
    assert flce.flce_linear_fp4_workspace_size(-1, 2048, 124160) == 0
