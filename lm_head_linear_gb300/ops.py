"""The operators around the LM head: the norm in front of it (and with its input
kept in 8 bits for the backward), its product with 8-bit and with 4-bit weights, drawing
tokens from logits, and the policy and preference losses on the log-probabilities
it returns.

As in :mod:`.binding`, arguments are checked, outputs and workspaces allocated
with torch (or taken from the caller), and the library's kernels do the work.
These calls are a few microseconds long on the GPU, so the checking and calling is
compiled (``csrc/ops_binding.cpp``, built into ``_lib/flce_ops.so``); there is no
fallback for it.
"""

from __future__ import annotations

import importlib.util
import os
from typing import Optional

import torch

from .binding import LIB_PATH, REDUCTIONS, _check, first_order, load_library

OPS_PATH = os.path.join(os.path.dirname(LIB_PATH), "flce_ops.so")
_OPS = None


def load_operators():
    """The compiled module (raises if it was not built)."""
    global _OPS
    if _OPS is None:
        load_library()
        if not os.path.exists(OPS_PATH):
            raise RuntimeError(f"{OPS_PATH} is missing: build it with `python -m lm_head_linear_gb300.build` "
                               "(there is no fallback implementation)")
        from .build import ops_built_for, running  # here: `python -m` runs that module itself
        if ops_built_for() != running():
            raise RuntimeError(f"{OPS_PATH} was built for {ops_built_for() or 'an unknown torch'}, this is {running()}: "
                               "build it again with `python -m lm_head_linear_gb300.build`")
        spec = importlib.util.spec_from_file_location("flce_ops", OPS_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.set_check(_check)
        _OPS = module
    return _OPS


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
    return (_OPS or load_operators()).add_rms_norm(x, weight, residual, eps, normed, fp8, save_rstd, stream, out)


def flce_add_rms_norm_backward_workspace_size(T: int, Hd: int) -> int:
    return int(load_library().flce_add_rms_norm_backward_workspace_size(T, Hd))


def flce_add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                               dh: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                               stream=None, out: Optional[dict] = None):
    """Run ``flce_add_rms_norm_backward``; returns ``(dx [T, Hd] in h's dtype, dweight [Hd] fp32, workspace)``.
    ``dx`` is the gradient of x and of the residual; ``dh`` an upstream gradient on h.
    ``out`` may hold preallocated ``dx`` and ``dweight`` tensors."""
    return (_OPS or load_operators()).add_rms_norm_backward(dy, h, weight, rstd, dh, workspace, stream, out)


def flce_add_rms_norm_checkpoint(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                                 eps: float = 1e-6, stream=None, out: Optional[dict] = None):
    """Run ``flce_add_rms_norm_checkpoint``; returns ``(y, h, rstd, hq, hq_scale)``: what :func:`flce_add_rms_norm`
    returns as y, h and rstd, and h in 8 bits for the backward (``hq`` float8_e4m3fn [T, Hd], ``hq_scale``
    float8_e8m0fnu per 128 channels).  ``out`` may hold preallocated tensors under those names."""
    return (_OPS or load_operators()).add_rms_norm_checkpoint(x, weight, residual, eps, stream, out)


def flce_add_rms_norm_checkpoint_backward(dy: torch.Tensor, hq: torch.Tensor, hq_scale: torch.Tensor, weight: torch.Tensor,
                                          rstd: torch.Tensor, dh: Optional[torch.Tensor] = None,
                                          dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                                          stream=None, out: Optional[dict] = None):
    """Run ``flce_add_rms_norm_checkpoint_backward``; returns ``(dx [T, Hd] in ``dtype``, dweight [Hd] fp32, workspace)``.
    ``dtype`` is h's (bfloat16 or float32), and ``dh``'s where that is given; the workspace has
    :func:`flce_add_rms_norm_backward_workspace_size` bytes.  ``out`` may hold preallocated ``dx`` and ``dweight``."""
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("dtype must be bfloat16 or float32")
    return (_OPS or load_operators()).add_rms_norm_checkpoint_backward(dy, hq, hq_scale, weight, rstd, dh,
                                                                       dtype is torch.float32, workspace, stream, out)


class AddRMSNorm(torch.autograd.Function):
    """autograd wrapper of the norm: returns ``(y, h)``, both differentiable."""

    @staticmethod
    def forward(ctx, x, weight, residual=None, eps: float = 1e-6, checkpoint: bool = False):
        if checkpoint:
            y, h, rstd, hq, hq_scale = flce_add_rms_norm_checkpoint(x, weight, residual, eps)
            ctx.save_for_backward(hq, hq_scale, weight, rstd)
        else:
            y, h, rstd, _, _ = flce_add_rms_norm(x, weight, residual, eps, save_rstd=True)
            ctx.save_for_backward(h, weight, rstd)
        ctx.checkpoint, ctx.h_dtype = checkpoint, h.dtype
        ctx.x_dtype = x.dtype
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        if residual is None:
            h = x.view_as(x)  # an input returned as it is would lose its place in the graph
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        if dy is not None:
            return AddRMSNorm._through_the_norm(ctx, dy, dh)
        if dh is None:
            return None, None, None, None, None
        return dh.to(ctx.x_dtype), None, dh if ctx.has_residual else None, None, None

    @staticmethod
    @first_order
    def _through_the_norm(ctx, dy, dh):
        dh = None if dh is None else _dense_rows(dh.to(ctx.h_dtype))
        if ctx.checkpoint:
            hq, hq_scale, weight, rstd = ctx.saved_tensors
            dx, dw, _ = flce_add_rms_norm_checkpoint_backward(_dense_rows(dy), hq, hq_scale, weight, rstd, dh=dh,
                                                              dtype=ctx.h_dtype)
        else:
            h, weight, rstd = ctx.saved_tensors
            dx, dw, _ = flce_add_rms_norm_backward(_dense_rows(dy), h, weight, rstd, dh=dh)
        return dx.to(ctx.x_dtype), dw.to(weight.dtype), dx if ctx.has_residual else None, None, None


def _dense_rows(t: torch.Tensor) -> torch.Tensor:
    """A gradient as the kernels take it (expanded, transposed and misaligned ones are copied)."""
    return t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] and t.data_ptr() % 16 == 0 and \
        t.stride(0) * t.element_size() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def add_rms_norm(x, weight, residual=None, eps: float = 1e-6, checkpoint: bool = False):
    """``(rms_norm(x + residual) * weight, x + residual)``, differentiable in every input.  With ``checkpoint`` the
    graph holds x + residual in 8 bits (one byte a channel and a scale per 128) instead of as it is; the forward is
    the same, and the gradients are those at the rounded values."""
    return AddRMSNorm.apply(x, weight, residual, eps, checkpoint)


def flce_quantize_fp8(a: torch.Tensor, block_rows: int = 128, stream=None, out: Optional[dict] = None):
    """Run ``flce_quantize_fp8``; returns ``(q float8_e4m3fn [rows, K], q_scale float8_e8m0fnu)``: one scale
    per ``block_rows`` x 128 block, 128 for weights, 1 for activations.  ``out`` may hold preallocated
    ``q`` and ``q_scale`` tensors."""
    return (_OPS or load_operators()).quantize_fp8(a, block_rows, stream, out)


def flce_linear_fp8_workspace_size(T: int, K: int, V: int) -> int:
    return int(load_library().flce_linear_fp8_workspace_size(T, K, V))


def flce_linear_fp8(x: torch.Tensor, x_scale: torch.Tensor, W: torch.Tensor, W_scale: torch.Tensor,
                    dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None, stream=None,
                    out: Optional[dict] = None):
    """Run ``flce_linear_fp8``; returns ``(y [T, V], workspace)`` in ``dtype`` (bfloat16 or float32).

    ``x`` [T, K] and ``W`` [V, K] are float8_e4m3fn with one E8M0 scale (float8_e8m0fnu, or
    its bytes as uint8) per row and 128 channels (``x_scale`` [T, ceil(K/128)]) and per 128 x
    128 block (``W_scale``): what :func:`flce_add_rms_norm` and :func:`flce_quantize_fp8`
    write.  ``out`` may hold a preallocated ``y``, whose rows may be longer than V.
    """
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("dtype must be bfloat16 or float32")
    return (_OPS or load_operators()).linear_fp8(x, x_scale, W, W_scale, dtype is torch.float32, workspace, stream, out)


def flce_quantize_fp4(a: torch.Tensor, stream=None, out: Optional[dict] = None):
    """Run ``flce_quantize_fp4``; returns ``(q uint8 [rows, 64 kb], q_scale float8_e8m0fnu [kb, rows, 4])``,
    kb = ceil(K / 128): two e2m1 numbers to a byte, the first of two channels in its low bits, and one scale per
    row and 32 channels.  ``out`` may hold preallocated ``q`` and ``q_scale`` tensors."""
    return (_OPS or load_operators()).quantize_fp4(a, stream, out)


def flce_linear_fp4_workspace_size(T: int, K: int, V: int) -> int:
    return int(load_library().flce_linear_fp4_workspace_size(T, K, V))


def flce_linear_fp4(x: torch.Tensor, x_scale: torch.Tensor, W: torch.Tensor, W_scale: torch.Tensor,
                    dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None, stream=None,
                    out: Optional[dict] = None):
    """Run ``flce_linear_fp4``; returns ``(y [T, V], workspace)`` in ``dtype`` (bfloat16 or float32).

    ``x`` and ``x_scale`` as :func:`flce_linear_fp8` takes them; ``W`` [V, 64 kb] uint8 and ``W_scale`` [kb, V, 4]
    (float8_e8m0fnu, or its bytes as uint8) as :func:`flce_quantize_fp4` writes them.  Packed weights that come
    with scales [V, 4 kb] need those laid out once: ``W_scale.view(V, kb, 4).transpose(0, 1).contiguous()``.
    ``out`` may hold a preallocated ``y``, whose rows may be longer than V.
    """
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("dtype must be bfloat16 or float32")
    return (_OPS or load_operators()).linear_fp4(x, x_scale, W, W_scale, dtype is torch.float32, workspace, stream, out)


def flce_sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, ignore_index: int = -100,
                stream=None, out: Optional[dict] = None):
    """Run ``flce_sample``; returns ``(tokens int64 [T], logp fp32 [T])``: one token drawn for each row of
    ``logits`` [T, V] (bfloat16 or float32, rows at any distance) with the random numbers ``u`` [T] (float32 in
    [0, 1)), and the log of the probability it was drawn with.

    ``temperature``, ``top_p``, ``min_p`` (float32) and ``top_k`` (int32) are numbers for all rows or tensors [T].
    Temperature 0 draws the largest logit of the lowest index; top_k 0, top_p 1 and min_p 0 keep every word.  Infinite
    temperatures are taken from a tensor only.  Logits
    of -inf are never drawn; a row of nothing else gets the token ``ignore_index``, which the losses leave out.  ``out``
    may hold preallocated ``tokens`` and ``logp`` tensors.
    """
    return (_OPS or load_operators()).sample(logits, u, temperature, top_k, top_p, min_p, ignore_index, stream, out)


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
    return (_OPS or load_operators()).policy_loss(logp, old_logp, advantages, targets, ref_logp, cu_seqlens, per_sequence,
                                        ignore_index, POLICY_REDUCTIONS[reduction], clip_low, clip_high, dual_clip,
                                        kl_coef, KL_KINDS[kl], dloss, forward, grad, workspace, stream, out)


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
    @first_order
    def backward(ctx, dloss, _):
        logp, old_logp, advantages, targets, ref_logp, cu_seqlens = ctx.saved_tensors
        _, dlogp, _, _, _ = flce_policy_loss(logp, old_logp, advantages, targets, ref_logp=ref_logp,
                                             cu_seqlens=cu_seqlens, dloss=dloss.contiguous(), forward=False,
                                             **ctx.kwargs)
        return dlogp, None, None, None, None, None, None


def policy_loss(logp, old_logp, advantages, targets, ref_logp=None, cu_seqlens=None, workspace=None, **kwargs):
    """Clipped policy loss with a KL term, differentiable in ``logp``; returns ``(loss, stats)``.
    Keyword arguments as :func:`flce_policy_loss` (per_sequence, ignore_index, reduction, clip_low,
    clip_high, dual_clip, kl_coef, kl).

    Malformed ``cu_seqlens`` are found on the GPU and make the results mean nothing: pass a ``workspace`` (uint8,
    :func:`flce_policy_loss_workspace_size` bytes) and look at it with :func:`.binding.flce_read_device_status`, which
    waits for the GPU.  Forward and backward both use it and leave their status there."""
    return PolicyLoss.apply(logp, old_logp, advantages, targets, ref_logp, cu_seqlens, dict(kwargs, workspace=workspace))


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
    return (_OPS or load_operators()).preference_loss(logp, targets, cu_seqlens, ref_logp, ignore_index, REDUCTIONS[reduction],
                                            PREFERENCE_KINDS[kind], beta, label_smoothing, margin, length_normalize,
                                            dloss, forward, grad, workspace, stream, out)


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
    @first_order
    def backward(ctx, dloss, _c, _r):
        logp, targets, cu_seqlens, ref_logp = ctx.saved_tensors
        _, dlogp, _, _, _ = flce_preference_loss(logp, targets, cu_seqlens, ref_logp=ref_logp,
                                                 dloss=dloss.contiguous(), forward=False, **ctx.kwargs)
        return dlogp, None, None, None, None


def preference_loss(logp, targets, cu_seqlens, ref_logp=None, workspace=None, **kwargs):
    """Preference loss on paired log ratios, differentiable in ``logp``; returns
    ``(loss, chosen_rewards, rejected_rewards)``.  Keyword arguments as
    :func:`flce_preference_loss` (ignore_index, reduction, kind, beta, label_smoothing, margin,
    length_normalize); ``workspace`` (:func:`flce_preference_loss_workspace_size` bytes) as in :func:`policy_loss`."""
    return PreferenceLoss.apply(logp, targets, cu_seqlens, ref_logp, dict(kwargs, workspace=workspace))
