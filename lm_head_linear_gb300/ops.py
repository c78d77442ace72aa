"""The operators around the LM head: the norm in front of it, its
product in 8 bits, and the policy and preference losses on the log-probabilities
it returns.

As in :mod:`.binding`: arguments are checked, outputs and workspaces allocated
with torch (or taken from the caller), and the library's kernels do the work.
These calls can be a few microseconds long on the GPU, so their Python side is
kept short: pointers go to ctypes as plain integers.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import binding
from .binding import REDUCTIONS, _check, load_library

_DTYPES = {torch.bfloat16: 0, torch.float32: 1}  # flce_dtype
_F32, _I64 = torch.float32, torch.int64
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(stream, device) -> int:
    return _raw_stream(device.index) if stream is None else stream.cuda_stream


def _out(out: Optional[dict], key: str, shape, dtype, device) -> torch.Tensor:
    """A new tensor, or the caller's out[key], checked."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return binding._out(out, key, shape, dtype, device)


def _rows(name: str, t: torch.Tensor, shape, device, dtypes=_DTYPES) -> int:
    """Checks a [T, Hd] tensor with contiguous rows; returns its row stride in elements."""
    ld, step = t.stride() if t.dim() == 2 else (0, 0)
    if t.dtype not in dtypes or t.shape != shape or t.device != device or step != 1:
        raise ValueError(f"{name} must be a {' or '.join(map(str, dtypes))} tensor of shape {tuple(shape)} on {device} "
                         f"with contiguous rows, got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")
    return ld if shape[0] > 1 else shape[1]


def _vector(name: str, t: torch.Tensor, n: int, dtype, device):
    if t.dtype is not dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _ws(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    if workspace.device != device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous uint8 tensor on {device}")
    return workspace


def _weight(weight: torch.Tensor, Hd: int, device) -> int:
    if weight.dtype not in _DTYPES or weight.shape != (Hd,) or weight.device != device or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous bfloat16 or float32 tensor of {Hd} elements on {device}")
    return _DTYPES[weight.dtype]


def flce_add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, normed: bool = True, fp8: bool = False, save_rstd: bool = False, stream=None,
                      out: Optional[dict] = None):
    """Run ``flce_add_rms_norm``; returns ``(y, h, rstd, q, q_scale)``.

    ``h`` is x + residual in the residual's dtype (x itself without a residual);
    ``y`` the bf16 norm (with ``normed``), ``q`` / ``q_scale`` its e4m3 form with a
    float8_e8m0fnu scale per 128 channels (with ``fp8``), ``rstd`` with
    ``save_rstd``; None where not asked for.  ``out`` may hold preallocated tensors
    under those names (``h`` may be the residual).
    """
    if not x.is_cuda or x.dim() != 2:
        raise ValueError("x must be a CUDA tensor [T, Hd]")
    lib = load_library()
    dev, shape = x.device, x.shape
    T, Hd = shape
    ldx = _rows("x", x, shape, dev)
    w_dtype = _weight(weight, Hd, dev)
    h, ldr, ldh, r_dtype = x, 0, 0, 0
    if residual is not None:
        ldr = _rows("residual", residual, shape, dev)
        r_dtype = _DTYPES[residual.dtype]
        h = (out or {}).get("h")
        if h is None:
            h = torch.empty(shape, dtype=residual.dtype, device=dev)
        ldh = _rows("out['h']", h, shape, dev, (residual.dtype,))
    y = _out(out, "y", shape, torch.bfloat16, dev) if normed else None
    rstd = _out(out, "rstd", T, _F32, dev) if save_rstd else None
    q = _out(out, "q", shape, torch.float8_e4m3fn, dev) if fp8 else None
    qs = _out(out, "q_scale", (T, (Hd + 127) // 128), torch.float8_e8m0fnu, dev) if fp8 else None
    _check(lib.flce_add_rms_norm(
        x.data_ptr(), _DTYPES[x.dtype], ldx, residual.data_ptr() if residual is not None else None, r_dtype, ldr,
        weight.data_ptr(), w_dtype, T, Hd, eps, h.data_ptr() if residual is not None else None, ldh,
        y.data_ptr() if normed else None, rstd.data_ptr() if save_rstd else None, q.data_ptr() if fp8 else None,
        qs.data_ptr() if fp8 else None, _stream(stream, dev)))
    return y, h, rstd, q, qs


def flce_add_rms_norm_backward_workspace_size(T: int, Hd: int) -> int:
    return int(load_library().flce_add_rms_norm_backward_workspace_size(T, Hd))


def flce_add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                               dh: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                               stream=None, out: Optional[dict] = None):
    """Run ``flce_add_rms_norm_backward``; returns ``(dx [T, Hd] in h's dtype, dweight [Hd] fp32, workspace)``.
    ``dx`` is the gradient of x and of the residual; ``dh`` an upstream gradient on h.
    ``out`` may hold preallocated ``dx`` and ``dweight`` tensors."""
    if not h.is_cuda or h.dim() != 2:
        raise ValueError("h must be a CUDA tensor [T, Hd]")
    lib = load_library()
    dev, shape = h.device, h.shape
    T, Hd = shape
    ldh = _rows("h", h, shape, dev)
    lddy = _rows("dy", dy, shape, dev)
    w_dtype = _weight(weight, Hd, dev)
    _vector("rstd", rstd, T, _F32, dev)
    lddh = _rows("dh", dh, shape, dev, (h.dtype,)) if dh is not None else 0
    dx = _out(out, "dx", shape, h.dtype, dev)
    dw = _out(out, "dweight", Hd, _F32, dev)
    ws = _ws(lib.flce_add_rms_norm_backward_workspace_size(T, Hd), dev, workspace)
    _check(lib.flce_add_rms_norm_backward(
        dy.data_ptr(), _DTYPES[dy.dtype], lddy, h.data_ptr(), _DTYPES[h.dtype], ldh, weight.data_ptr(), w_dtype,
        rstd.data_ptr(), dh.data_ptr() if dh is not None else None, lddh, T, Hd, dx.data_ptr(), dw.data_ptr(),
        ws.data_ptr(), ws.numel(), _stream(stream, dev)))
    return dx, dw, ws


class AddRMSNorm(torch.autograd.Function):
    """autograd wrapper of the norm: returns ``(y, h)``, both differentiable."""

    @staticmethod
    def forward(ctx, x, weight, residual=None, eps: float = 1e-6):
        y, h, rstd, _, _ = flce_add_rms_norm(x, weight, residual, eps, save_rstd=True)
        ctx.save_for_backward(h, weight, rstd)
        ctx.x_dtype = x.dtype
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        if residual is None:
            h = x.view_as(x)  # an input returned as it is would lose its place in the graph
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, weight, rstd = ctx.saved_tensors
        if dy is None and dh is None:
            return None, None, None, None
        if dy is None:
            dx, dw = dh, None
        else:
            dx, dw, _ = flce_add_rms_norm_backward(_dense_rows(dy), h, weight, rstd,
                                                   dh=None if dh is None else _dense_rows(dh.to(h.dtype)))
            dw = dw.to(weight.dtype)
        return dx.to(ctx.x_dtype), dw, dx if ctx.has_residual else None, None


def _dense_rows(t: torch.Tensor) -> torch.Tensor:
    """A gradient as the kernels take it (expanded and transposed ones are copied)."""
    return t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] and t.data_ptr() % 16 == 0 and \
        t.stride(0) * t.element_size() % 16 == 0 else t.contiguous()


def add_rms_norm(x, weight, residual=None, eps: float = 1e-6):
    """``(rms_norm(x + residual) * weight, x + residual)``, differentiable in every input."""
    return AddRMSNorm.apply(x, weight, residual, eps)


# Scales are E8M0 bytes: torch's float8_e8m0fnu, or the bytes as uint8.
_SCALES = (torch.float8_e8m0fnu, torch.uint8)


def _blocks(name: str, q: torch.Tensor, scale: torch.Tensor, block_rows: int, device):
    if q.dtype != torch.float8_e4m3fn or q.dim() != 2 or q.device != device or not q.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float8_e4m3fn matrix on {device}")
    want = ((q.shape[0] + block_rows - 1) // block_rows, (q.shape[1] + 127) // 128)
    if scale.dtype not in _SCALES or scale.shape != want or scale.device != device or not scale.is_contiguous():
        raise ValueError(f"{name}'s scales must be a contiguous float8_e8m0fnu or uint8 tensor of shape {want} on {device}, "
                         f"got {scale.dtype} {tuple(scale.shape)} on {scale.device}")


def flce_quantize_fp8(a: torch.Tensor, block_rows: int = 128, stream=None, out: Optional[dict] = None):
    """Run ``flce_quantize_fp8``; returns ``(q float8_e4m3fn [rows, K], q_scale float8_e8m0fnu)``: one scale
    per ``block_rows`` x 128 block, 128 for weights, 1 for activations.  ``out`` may hold preallocated
    ``q`` and ``q_scale`` tensors."""
    if not a.is_cuda or a.dim() != 2:
        raise ValueError("a must be a CUDA matrix")
    dev, (rows, K) = a.device, a.shape
    lda = _rows("a", a, a.shape, dev)
    q = _out(out, "q", (rows, K), torch.float8_e4m3fn, dev)
    qs = _out(out, "q_scale", ((rows + block_rows - 1) // max(block_rows, 1), (K + 127) // 128), torch.float8_e8m0fnu, dev)
    _check(load_library().flce_quantize_fp8(a.data_ptr(), _DTYPES[a.dtype], lda, rows, K, block_rows, q.data_ptr(),
                                            qs.data_ptr(), _stream(stream, dev)))
    return q, qs


def flce_linear_fp8_workspace_size(T: int, K: int, V: int) -> int:
    return int(load_library().flce_linear_fp8_workspace_size(T, K, V))


def flce_linear_fp8(x: torch.Tensor, x_scale: torch.Tensor, W: torch.Tensor, W_scale: torch.Tensor,
                    dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None, stream=None,
                    out: Optional[dict] = None):
    """Run ``flce_linear_fp8``; returns ``(y [T, V], workspace)`` in ``dtype`` (bfloat16 or float32).

    ``x`` [T, K] and ``W`` [V, K] are float8_e4m3fn with one E8M0 scale per row and 128
    channels (``x_scale`` [T, ceil(K/128)]) and per 128 x 128 block (``W_scale``): what
    :func:`flce_add_rms_norm` and :func:`flce_quantize_fp8` write.  ``out`` may hold a
    preallocated ``y``, whose rows may be longer than V.
    """
    if not x.is_cuda or x.dim() != 2 or W.dim() != 2 or W.shape[1] != x.shape[1]:
        raise ValueError("x [T, K] and W [V, K] must be CUDA matrices of equal K")
    lib = load_library()
    dev, (T, K), V = x.device, x.shape, W.shape[0]
    _blocks("x", x, x_scale, 1, dev)
    _blocks("W", W, W_scale, 128, dev)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be bfloat16 or float32")
    y = (out or {}).get("y")
    if y is None:
        y = torch.empty((T, V), dtype=dtype, device=dev)
    ldy = _rows("out['y']", y, torch.Size((T, V)), dev, (dtype,))
    ws = _ws(256, dev, workspace)
    _check(lib.flce_linear_fp8(x.data_ptr(), x_scale.data_ptr(), W.data_ptr(), W_scale.data_ptr(), T, K, V, y.data_ptr(),
                               _DTYPES[dtype], ldy, ws.data_ptr(), ws.numel(), _stream(stream, dev)))
    return y, ws


POLICY_REDUCTIONS = {"none": 0, "mean": 1, "sum": 2, "sequence_mean": 3}
KL_KINDS = {"k1": 1, "k2": 2, "k3": 3}
PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}


def flce_policy_loss_workspace_size(T: int, n_seqs: int) -> int:
    return int(load_library().flce_policy_loss_workspace_size(T, n_seqs))


def flce_policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, targets: torch.Tensor,
                     ref_logp: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                     per_sequence: bool = False, ignore_index: int = -100, reduction: str = "mean",
                     clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: float = 0.0, kl_coef: float = 0.0,
                     kl: str = "k3", dloss: Optional[torch.Tensor] = None, forward: bool = True, grad: bool = True,
                     workspace: Optional[torch.Tensor] = None, stream=None, out: Optional[dict] = None):
    """Run ``flce_policy_loss``; returns ``(loss, dlogp, stats, n_valid, workspace)``.

    ``loss`` is a 1-element fp32 tensor ([T] with reduction "none"; None without
    ``forward``), ``dlogp`` the gradient on logp, already multiplied with ``dloss``
    (None without ``grad``): pass it to :func:`flce_backward` as ``dlogp``.  ``stats``
    holds the valid tokens' means of (kl, clipped, log ratio, ratio).  ``advantages``
    is [T], or with ``per_sequence`` one per sequence of ``cu_seqlens``.  ``out`` may
    hold preallocated ``loss``, ``dlogp``, ``stats`` and ``n_valid`` tensors.
    """
    if not logp.is_cuda or logp.dim() != 1:
        raise ValueError("logp must be a CUDA tensor [T]")
    lib = load_library()
    dev, T = logp.device, logp.shape[0]
    red = POLICY_REDUCTIONS[reduction]
    n_seqs = 0
    if cu_seqlens is not None:
        n_seqs = cu_seqlens.shape[0] - 1 if cu_seqlens.dim() == 1 else -1
        if n_seqs < 0:
            raise ValueError("cu_seqlens must be a tensor [n_seqs + 1]")
        _vector("cu_seqlens", cu_seqlens, n_seqs + 1, _I64, dev)
    _vector("logp", logp, T, _F32, dev)
    _vector("old_logp", old_logp, T, _F32, dev)
    _vector("advantages", advantages, n_seqs if per_sequence else T, _F32, dev)
    _vector("targets", targets, T, _I64, dev)
    if ref_logp is not None:
        _vector("ref_logp", ref_logp, T, _F32, dev)
    if dloss is not None:
        dloss = dloss.reshape(-1)
        _vector("dloss", dloss, T if red == 0 else 1, _F32, dev)
    loss = _out(out, "loss", T if red == 0 else 1, _F32, dev) if forward else None
    dlogp = _out(out, "dlogp", T, _F32, dev) if grad else None
    stats = _out(out, "stats", 4, _F32, dev)
    n_valid = _out(out, "n_valid", 1, _I64, dev)
    ws = _ws(lib.flce_policy_loss_workspace_size(T, n_seqs), dev, workspace)
    _check(lib.flce_policy_loss(
        dloss.data_ptr() if dloss is not None else None, logp.data_ptr(), old_logp.data_ptr(),
        ref_logp.data_ptr() if ref_logp is not None else None, advantages.data_ptr(), per_sequence, targets.data_ptr(),
        cu_seqlens.data_ptr() if cu_seqlens is not None else None, n_seqs, T, ignore_index, red, clip_low, clip_high,
        dual_clip, kl_coef, KL_KINDS[kl], loss.data_ptr() if forward else None, dlogp.data_ptr() if grad else None,
        stats.data_ptr(), n_valid.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream, dev)))
    return loss, dlogp, stats, n_valid, ws


class PolicyLoss(torch.autograd.Function):
    """autograd wrapper of the policy loss, differentiable in logp."""

    @staticmethod
    def forward(ctx, logp, old_logp, advantages, targets, ref_logp, cu_seqlens, kwargs):
        logp = logp.contiguous()
        loss, _, stats, _, ws = flce_policy_loss(logp, old_logp, advantages, targets, ref_logp=ref_logp,
                                                 cu_seqlens=cu_seqlens, grad=False, **kwargs)
        ctx.save_for_backward(logp, old_logp, advantages, targets, ref_logp, cu_seqlens)
        ctx.kwargs = kwargs
        ctx.mark_non_differentiable(stats)
        return (loss if kwargs.get("reduction") == "none" else loss.reshape(())), stats

    @staticmethod
    def backward(ctx, dloss, _):
        logp, old_logp, advantages, targets, ref_logp, cu_seqlens = ctx.saved_tensors
        _, dlogp, _, _, _ = flce_policy_loss(logp, old_logp, advantages, targets, ref_logp=ref_logp,
                                             cu_seqlens=cu_seqlens, dloss=dloss.contiguous(), forward=False,
                                             **ctx.kwargs)
        return dlogp, None, None, None, None, None, None


def policy_loss(logp, old_logp, advantages, targets, ref_logp=None, cu_seqlens=None, **kwargs):
    """Clipped policy loss with a KL term, differentiable in ``logp``; returns ``(loss, stats)``.
    Keyword arguments as :func:`flce_policy_loss` (per_sequence, ignore_index, reduction, clip_low,
    clip_high, dual_clip, kl_coef, kl)."""
    return PolicyLoss.apply(logp, old_logp, advantages, targets, ref_logp, cu_seqlens, kwargs)


def flce_preference_loss_workspace_size(n_pairs: int) -> int:
    return int(load_library().flce_preference_loss_workspace_size(n_pairs))


def flce_preference_loss(logp: torch.Tensor, targets: torch.Tensor, cu_seqlens: torch.Tensor,
                         ref_logp: Optional[torch.Tensor] = None, ignore_index: int = -100, reduction: str = "mean",
                         kind: str = "sigmoid", beta: float = 0.1, label_smoothing: float = 0.0, margin: float = 0.0,
                         length_normalize: bool = False, dloss: Optional[torch.Tensor] = None, forward: bool = True,
                         grad: bool = True, workspace: Optional[torch.Tensor] = None, stream=None,
                         out: Optional[dict] = None):
    """Run ``flce_preference_loss``; returns ``(loss, dlogp, chosen_rewards, rejected_rewards, workspace)``.

    ``cu_seqlens`` [2 P + 1]: sequence 2p is pair p's chosen answer, 2p + 1 the rejected
    one.  ``loss`` is a 1-element fp32 tensor ([P] with reduction "none"; None without
    ``forward``), ``dlogp`` [T] the gradient on logp, already multiplied with ``dloss``
    (None without ``grad``).  ``out`` may hold preallocated ``loss``, ``dlogp``, ``chosen``
    and ``rejected`` tensors.
    """
    if not logp.is_cuda or logp.dim() != 1:
        raise ValueError("logp must be a CUDA tensor [T]")
    lib = load_library()
    dev, T = logp.device, logp.shape[0]
    red = REDUCTIONS[reduction]
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] % 2 == 0:
        raise ValueError("cu_seqlens must be a tensor [2 n_pairs + 1]")
    P = cu_seqlens.shape[0] // 2
    _vector("cu_seqlens", cu_seqlens, 2 * P + 1, _I64, dev)
    _vector("logp", logp, T, _F32, dev)
    _vector("targets", targets, T, _I64, dev)
    if ref_logp is not None:
        _vector("ref_logp", ref_logp, T, _F32, dev)
    if dloss is not None:
        dloss = dloss.reshape(-1)
        _vector("dloss", dloss, P if red == 0 else 1, _F32, dev)
    loss = _out(out, "loss", P if red == 0 else 1, _F32, dev) if forward else None
    dlogp = _out(out, "dlogp", T, _F32, dev) if grad else None
    chosen = _out(out, "chosen", P, _F32, dev)
    rejected = _out(out, "rejected", P, _F32, dev)
    ws = _ws(lib.flce_preference_loss_workspace_size(P), dev, workspace)
    _check(lib.flce_preference_loss(
        dloss.data_ptr() if dloss is not None else None, logp.data_ptr(),
        ref_logp.data_ptr() if ref_logp is not None else None, targets.data_ptr(), cu_seqlens.data_ptr(), P, T,
        ignore_index, red, PREFERENCE_KINDS[kind], beta, label_smoothing, margin, length_normalize,
        loss.data_ptr() if forward else None, dlogp.data_ptr() if grad else None, chosen.data_ptr(),
        rejected.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream, dev)))
    return loss, dlogp, chosen, rejected, ws


class PreferenceLoss(torch.autograd.Function):
    """autograd wrapper of the preference loss, differentiable in logp."""

    @staticmethod
    def forward(ctx, logp, targets, cu_seqlens, ref_logp, kwargs):
        logp = logp.contiguous()
        loss, _, chosen, rejected, _ = flce_preference_loss(logp, targets, cu_seqlens, ref_logp=ref_logp, grad=False,
                                                            **kwargs)
        ctx.save_for_backward(logp, targets, cu_seqlens, ref_logp)
        ctx.kwargs = kwargs
        ctx.mark_non_differentiable(chosen, rejected)
        return (loss if kwargs.get("reduction") == "none" else loss.reshape(())), chosen, rejected

    @staticmethod
    def backward(ctx, dloss, _c, _r):
        logp, targets, cu_seqlens, ref_logp = ctx.saved_tensors
        _, dlogp, _, _, _ = flce_preference_loss(logp, targets, cu_seqlens, ref_logp=ref_logp,
                                                 dloss=dloss.contiguous(), forward=False, **ctx.kwargs)
        return dlogp, None, None, None, None


def preference_loss(logp, targets, cu_seqlens, ref_logp=None, **kwargs):
    """Preference loss on paired log ratios, differentiable in ``logp``; returns
    ``(loss, chosen_rewards, rejected_rewards)``.  Keyword arguments as
    :func:`flce_preference_loss` (ignore_index, reduction, kind, beta, label_smoothing, margin,
    length_normalize)."""
    return PreferenceLoss.apply(logp, targets, cu_seqlens, ref_logp, kwargs)
