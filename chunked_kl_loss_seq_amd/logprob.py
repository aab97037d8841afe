"""Log-probabilities of given tokens with entropy, and the most likely
alternatives: from logits, and from hidden states under the head's weight without
ever holding their logits; with gradients.

Argument checks and marshalling only, as in ``binding``: every step runs in the
library's HIP kernels on the current stream of the tensors' device, and CPU
tensors raise.
"""
from __future__ import annotations

import ctypes
from typing import Any, NamedTuple

from .binding import DTYPE_BF16, DTYPE_F32, _check, _check_out, lib
from .residual import _at, _call, _no_capture
from .vocab import _dtype, _gpu


class LogProbs(NamedTuple):
    """What ``logprobs`` gives: logp float32 like ids (None without ids), entropy
    float32 [N], stats float32 [2, N] (a row's largest logit and the log of the sum
    of exp(z - largest), together its log-normaliser), and the alternatives' ids
    int32 [N, top] and log-probabilities float32 [N, top] (None without)."""

    logp: Any
    entropy: Any
    stats: Any
    top_ids: Any
    top_logp: Any


class HeadLogProbs(NamedTuple):
    """What ``head_logprobs`` gives; see ``LogProbs``."""

    logp: Any
    entropy: Any
    stats: Any


def _given(torch, ids, mask, N, dev):
    """(T, mask as uint8) after checking the given tokens [N] or [N, T] and the mask [N]."""
    T = 0
    if ids is not None:
        if ids.dtype != torch.int32 or not ids.is_contiguous() or ids.device != dev:
            raise ValueError(f"ids must be a contiguous int32 tensor on {dev}")
        if ids.dim() not in (1, 2) or ids.shape[0] != N:
            raise ValueError("ids must be [N] or [N, T]")
        T = 1 if ids.dim() == 1 else ids.shape[1]
    if mask is not None:
        if tuple(mask.shape) != (N,) or mask.device != dev:
            raise ValueError(f"mask must be [N] on {dev}")
        mask = mask.contiguous()
        mask = mask.view(torch.uint8) if mask.dtype == torch.bool else mask.to(torch.uint8)
    return T, mask


def _upstream(torch, ids, T, dlogp, dentropy, N, dev):
    """Checks the gradients of logp (of the shape of ids) and of entropy."""
    if ids is None:
        if dlogp is not None:
            raise ValueError("dlogp needs ids")
    else:
        if dlogp is None:
            raise ValueError("dlogp must be given with ids")
        _check_out(torch, dlogp, tuple(ids.shape), torch.float32, dev, "dlogp")
    _check_out(torch, dentropy, (N,), torch.float32, dev, "dentropy")


def _logits(torch, logits):
    dev = _gpu(logits, "logits")
    dt = _dtype(torch, logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [N, V]")
    N, V = logits.shape
    if V > 1 and N > 0 and logits.stride(1) != 1:
        raise ValueError("the elements of a row of logits must be adjacent")
    return dev, dt, N, V, logits.stride(0) if N > 1 else V


def logprobs(logits, ids=None, top=0, mask=None):
    """Of each row of logits [N, V]: the log-probabilities of the given tokens ``ids``
    (int32 [N], or [N, T] with T up to 2,048), the entropy, and the ``top`` (up to
    512) most likely tokens with their log-probabilities, ordered as ``topk`` orders
    them: a ``LogProbs``.

    An id outside [0, V) is an entry without a token: log-probability 0.  ``mask``
    (uint8 or bool [N]): rows with 0 are not read, their results are 0 and their
    alternatives -1.  A logit of -inf has probability 0; a row of nothing else has
    entropy 0 and log-probabilities -inf, alternatives that are not there are -1 with
    -inf.  NaN or +inf in a row makes its log-probabilities and entropy NaN.

    logits are bfloat16 or float32 with adjacent elements in a row; rows may be
    strided (a slice of a padded vocabulary).
    """
    import torch

    dev, dt, N, V, ld = _logits(torch, logits)
    top = int(top)
    if not 0 <= top <= V:
        raise ValueError("top must be in 0 .. V")
    T, mask = _given(torch, ids, mask, N, dev)
    need = ctypes.c_uint64(0)
    _check(lib().ckl_logprobs_workspace(N, V, top, need), "ckl_logprobs_workspace")
    f32, empty = torch.float32, torch.empty
    logp = empty(*ids.shape, dtype=f32, device=dev) if ids is not None else None
    entropy = empty(N, dtype=f32, device=dev)
    stats = empty(2, N, dtype=f32, device=dev)
    top_ids = empty(N, top, dtype=torch.int32, device=dev) if top else None
    top_logp = empty(N, top, dtype=f32, device=dev) if top else None
    # from torch's allocator, so that calls on several streams, or captured into several graphs, never share it
    ws = empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
    _call(torch, dev, lib().ckl_logprobs, dt, logits.data_ptr(), N, V, ld, _at(ids), T, _at(mask), top, _at(logp),
          entropy.data_ptr(), stats.data_ptr(), _at(top_ids), _at(top_logp), _at(ws), need.value)
    return LogProbs(logp, entropy, stats, top_ids, top_logp)


def logprobs_bwd(logits, ids, entropy, stats, dlogp=None, dentropy=None, mask=None, out=None):
    """Gradient of ``logprobs`` with respect to the logits, in their type: [N, V].

    logits, ids and mask are the forward call's, entropy and stats its results; dlogp
    (float32, of the shape of ids) and dentropy (float32 [N], or None) the gradients
    of logp and entropy.  Entries without a token, masked rows and rows without any
    token of probability above 0 give nothing.  ``out`` may be the logits themselves.
    """
    import torch

    dev, dt, N, V, ld = _logits(torch, logits)
    T, mask = _given(torch, ids, mask, N, dev)
    _upstream(torch, ids, T, dlogp, dentropy, N, dev)
    if stats is None or (dentropy is not None and entropy is None):
        raise ValueError("logprobs_bwd needs the stats, and the entropy for its gradient, that logprobs returned")
    _check_out(torch, stats, (2, N), torch.float32, dev, "stats")
    _check_out(torch, entropy, (N,), torch.float32, dev, "entropy")
    if out is logits:
        ldo = ld
        if ldo < V:
            raise ValueError("logits whose rows overlap cannot be written to")
    else:
        _check_out(torch, out, (N, V), logits.dtype, dev, "out")
        ldo = V
    if out is None:
        out = torch.empty((N, V), dtype=logits.dtype, device=dev)
    _call(torch, dev, lib().ckl_logprobs_bwd, dt, logits.data_ptr(), N, V, ld, _at(ids), T, _at(mask), stats.data_ptr(),
          _at(entropy), _at(dlogp), _at(dentropy), out.data_ptr(), ldo)
    return out


class _TokenLogProbs:
    """torch.autograd.Function wrapper, created lazily so importing needs no torch."""

    _fn = None

    @classmethod
    def get(cls):
        if cls._fn is None:
            import torch

            class TokenLogProbs(torch.autograd.Function):
                @staticmethod
                def forward(ctx, logits, ids, mask):
                    if logits.dim() == 2 and logits.shape[1] > 1 and logits.stride(1) != 1:
                        logits = logits.contiguous()
                    out = logprobs(logits, ids, mask=mask)
                    ctx.save_for_backward(logits, ids, mask, out.entropy, out.stats)
                    ctx.set_materialize_grads(False)
                    return out.logp, out.entropy

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, dlogp, dentropy):
                    _no_capture(torch, "token_logprobs's backward", "logprobs and logprobs_bwd")
                    logits, ids, mask, entropy, stats = ctx.saved_tensors
                    if dlogp is None and dentropy is None:
                        return None, None, None
                    if dlogp is None and ids is not None:
                        ids = None  # the entropy's gradient alone
                    dlogp, dentropy = (None if g is None else g.contiguous() for g in (dlogp, dentropy))
                    return logprobs_bwd(logits, ids, entropy, stats, dlogp, dentropy, mask=mask), None, None

            cls._fn = TokenLogProbs
        return cls._fn


def token_logprobs(logits, ids, mask=None):
    """(log-probabilities of ids, entropy) of ``logprobs`` as a differentiable torch
    function of the logits.  A stream capture takes it only where no gradient is asked
    for; a captured training step calls ``logprobs`` and ``logprobs_bwd``."""
    import torch

    if logits.requires_grad and torch.is_grad_enabled():
        _no_capture(torch, "token_logprobs's forward", "logprobs and logprobs_bwd")
    return _TokenLogProbs.get().apply(logits, ids, mask)


def _head(torch, H, W):
    dev = _gpu(H, "H")
    dt = _dtype(torch, H, "H")
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1]:
        raise ValueError("H must be [N, d] and W [V, d]")
    if W.dtype != H.dtype or W.device != dev or not W.is_contiguous() or not H.is_contiguous():
        raise ValueError(f"H and W must be contiguous, of one type, on {dev}")
    return dev, dt, H.shape[0], H.shape[1], W.shape[0]


def head_logprobs_plan(N, d, V, dtype="bf16", backward=False, dw_dtype=None, chunk=0, budget_bytes=0):
    """(rows per chunk, workspace bytes) of ``head_logprobs`` or, with ``backward``, of
    ``head_logprobs_bwd`` with a dW of ``dw_dtype`` ("bf16" or "f32"; that of W if None)."""
    code = {"bf16": DTYPE_BF16, "f32": DTYPE_F32}
    c, b = ctypes.c_int64(0), ctypes.c_uint64(0)
    _check(lib().ckl_head_logprobs_plan(1 if backward else 0, code[dtype], code[dw_dtype or dtype], N, d, V, int(chunk),
                                        int(budget_bytes), ctypes.byref(c), ctypes.byref(b)), "ckl_head_logprobs_plan")
    return int(c.value), int(b.value)


def _plan(backward, dt, dw_dt, N, d, V, chunk):
    b = ctypes.c_uint64(0)
    _check(lib().ckl_head_logprobs_plan(backward, dt, dw_dt, N, d, V, chunk, 0, None, ctypes.byref(b)),
           "ckl_head_logprobs_plan")
    return b.value


def head_logprobs(H, W, ids=None, mask=None, chunk=0):
    """``logprobs`` of the logits H W^T, which are never held: a ``HeadLogProbs``.

    H [N, d] hidden states and W [V, d] the head's weight, both bfloat16 or both
    float32, contiguous, d a multiple of 8; ids and mask as for ``logprobs`` (masked
    positions cost no contraction).  Rows go in chunks whose workspace, from torch's
    allocator, keeps to CKL_WORKSPACE_BYTES (6 GiB if unset); ``chunk`` fixes their
    length.  Logits are fp32 sums and are not rounded.
    """
    import torch

    dev, dt, N, d, V = _head(torch, H, W)
    T, mask = _given(torch, ids, mask, N, dev)
    need = _plan(0, dt, 0, N, d, V, int(chunk))
    logp = torch.empty(ids.shape, dtype=torch.float32, device=dev) if ids is not None else None
    entropy = torch.empty((N,), dtype=torch.float32, device=dev)
    stats = torch.empty((2, N), dtype=torch.float32, device=dev)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(torch, dev, lib().ckl_head_logprobs, dt, H.data_ptr(), W.data_ptr(), _at(ids), _at(mask), N, d, V, T, int(chunk),
          _at(logp), entropy.data_ptr(), stats.data_ptr(), _at(ws), need)
    return HeadLogProbs(logp, entropy, stats)


def head_logprobs_bwd(H, W, ids, logp, entropy, stats, dlogp=None, dentropy=None, mask=None, chunk=0, dW=None,
                      accumulate=False):
    """Gradients of ``head_logprobs``: (dH like H, dW).

    The logits are recomputed.  H, W, ids and mask are the forward call's, logp,
    entropy and stats its results, dlogp (float32, of the shape of ids) and dentropy
    (float32 [N], or None) the gradients of logp and entropy.  dW has W's type, rounded
    once after the last chunk, or is the given tensor: of W's type or float32.  With
    ``accumulate`` the gradient is added to a given float32 dW, as ``fwd_bwd`` or
    ``bwd`` wrote it.
    """
    import torch

    dev, dt, N, d, V = _head(torch, H, W)
    T, mask = _given(torch, ids, mask, N, dev)
    _upstream(torch, ids, T, dlogp, dentropy, N, dev)
    if stats is None or (ids is not None and logp is None) or (dentropy is not None and entropy is None):
        raise ValueError("head_logprobs_bwd needs the logp, entropy and stats that head_logprobs returned")
    _check_out(torch, logp, tuple(ids.shape) if ids is not None else (), torch.float32, dev, "logp")
    _check_out(torch, entropy, (N,), torch.float32, dev, "entropy")
    _check_out(torch, stats, (2, N), torch.float32, dev, "stats")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs the dW to add to")
        dW = torch.empty((V, d), dtype=W.dtype, device=dev)
    if dW.dtype not in (W.dtype, torch.float32):
        raise ValueError("dW must have W's type or float32")
    if accumulate and dW.dtype != torch.float32:
        raise ValueError("accumulate needs a float32 dW")
    _check_out(torch, dW, (V, d), dW.dtype, dev, "dW")
    dw_dt = DTYPE_BF16 if dW.dtype == torch.bfloat16 else DTYPE_F32
    need = _plan(1, dt, dw_dt, N, d, V, int(chunk))
    dH = torch.empty_like(H)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(torch, dev, lib().ckl_head_logprobs_bwd, dt, H.data_ptr(), W.data_ptr(), _at(ids), _at(mask), N, d, V, T,
          int(chunk), _at(logp), _at(entropy), stats.data_ptr(), _at(dlogp), _at(dentropy), dH.data_ptr(), dw_dt,
          1 if accumulate else 0, dW.data_ptr(), _at(ws), need)
    return dH, dW


class _HeadTokenLogProbs:
    """torch.autograd.Function wrapper, created lazily so importing needs no torch."""

    _fn = None

    @classmethod
    def get(cls):
        if cls._fn is None:
            import torch

            class HeadTokenLogProbs(torch.autograd.Function):
                @staticmethod
                def forward(ctx, H, W, ids, mask, chunk):
                    H, W = H.contiguous(), W.contiguous()
                    out = head_logprobs(H, W, ids, mask, chunk)
                    ctx.save_for_backward(H, W, ids, mask, *out)
                    ctx.set_materialize_grads(False)
                    ctx.chunk = chunk
                    return out.logp, out.entropy

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, dlogp, dentropy):
                    _no_capture(torch, "head_token_logprobs's backward", "head_logprobs and head_logprobs_bwd")
                    H, W, ids, mask, logp, entropy, stats = ctx.saved_tensors
                    if dlogp is None and dentropy is None:
                        return (None,) * 5
                    if dlogp is None:
                        ids = logp = None  # the entropy's gradient alone
                    dlogp, dentropy = (None if g is None else g.contiguous() for g in (dlogp, dentropy))
                    dH, dW = head_logprobs_bwd(H, W, ids, logp, entropy, stats, dlogp, dentropy, mask, ctx.chunk)
                    return dH, dW, None, None, None

            cls._fn = HeadTokenLogProbs
        return cls._fn


def head_token_logprobs(H, W, ids, mask=None, chunk=0):
    """(log-probabilities of ids, entropy) of ``head_logprobs`` as a differentiable torch
    function of H and W (copied where they are not contiguous).  A stream capture takes
    it only where no gradient is asked for; a captured training step calls
    ``head_logprobs`` and ``head_logprobs_bwd``."""
    import torch

    if torch.is_grad_enabled() and (H.requires_grad or W.requires_grad):
        _no_capture(torch, "head_token_logprobs's forward", "head_logprobs and head_logprobs_bwd")
    return _HeadTokenLogProbs.get().apply(H, W, ids, mask, chunk)
