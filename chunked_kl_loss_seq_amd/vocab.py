"""Operators around the vocabulary table W [V, d], beside the loss at its head:
the embedding lookup and its gradient, and sampling tokens from logits.

Argument checks and marshalling only, as in ``binding``: every step runs in the
library's HIP kernels on the current stream of the tensors' device, and CPU
tensors raise.
"""
from __future__ import annotations

import contextlib
import ctypes

from .binding import DTYPE_BF16, DTYPE_F32, Sampling, _check, _check_out, _ptr, _stream, lib


def _dtype(torch, t, name):
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise ValueError(f"{name} must be bfloat16 or float32")


def _gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _on(torch, device):
    """The library launches on the current device: make it the tensors' one."""
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _check_ids(torch, ids, device):
    if ids.dtype != torch.int32 or not ids.is_contiguous() or ids.device != device:
        raise ValueError(f"ids must be a contiguous int32 tensor on {device}")


def embed(ids, W, scale=1.0, out=None):
    """scale x W[ids], rounded once to W's type: [..., d] for int32 ids of any shape.

    W [V, d] is bfloat16 or float32, contiguous, d a multiple of 8.  An id
    outside [0, V) is a position without a token (padding): its row is zeros.
    """
    import torch

    dev = _gpu(W, "W")
    dt = _dtype(torch, W, "W")
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous [V, d] tensor")
    _check_ids(torch, ids, dev)
    V, d = W.shape
    shape = (*ids.shape, d)
    _check_out(torch, out, shape, W.dtype, dev, "out")
    if out is None:
        out = torch.empty(shape, dtype=W.dtype, device=dev)
    with _on(torch, dev):
        _check(lib().ckl_embed(dt, _ptr(ids), _ptr(W), float(scale), ids.numel(), d, V, _ptr(out),
                               _stream(torch, dev)), "ckl_embed")
    return out


def embed_bwd(ids, dY, V, scale=1.0, dW=None, accumulate=False):
    """Gradient of ``embed`` with respect to W: float32 [V, d], the scaled sums of
    dY's rows by token, in a fixed order.

    dY [..., d] is bfloat16 or float32, contiguous, its leading shape that of
    the int32 ids.  With ``accumulate`` the sums are added to the given dW and
    rows of absent tokens are left alone: with tied weights, dW is then the
    head gradient that ``fwd_bwd`` or ``bwd`` wrote.
    """
    import torch

    dev = _gpu(dY, "dY")
    dt = _dtype(torch, dY, "dY")
    _check_ids(torch, ids, dev)
    if dY.dim() != ids.dim() + 1 or dY.shape[:-1] != ids.shape or not dY.is_contiguous():
        raise ValueError("dY must be contiguous, of the shape of ids and a last dimension d")
    N, d, V = ids.numel(), dY.shape[-1], int(V)
    _check_out(torch, dW, (V, d), torch.float32, dev, "dW")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs the dW to add to")
        dW = torch.empty((V, d), dtype=torch.float32, device=dev)
    need = ctypes.c_uint64(0)
    _check(lib().ckl_embed_bwd_workspace(N, d, V, ctypes.byref(need)), "ckl_embed_bwd_workspace")
    with _on(torch, dev):
        # from torch's allocator, so that calls on several streams, or captured
        # into several graphs, never share it
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
        _check(lib().ckl_embed_bwd(dt, _ptr(ids), _ptr(dY), float(scale), N, d, V, 1 if accumulate else 0, _ptr(dW),
                                   _ptr(ws), need.value, _stream(torch, dev)), "ckl_embed_bwd")
    return dW


class _Embedding:
    """torch.autograd.Function wrapper, created lazily so importing needs no torch."""

    _fn = None

    @classmethod
    def get(cls):
        if cls._fn is None:
            import torch

            class Embedding(torch.autograd.Function):
                @staticmethod
                def forward(ctx, ids, W, scale):
                    W = W.contiguous()
                    ctx.save_for_backward(ids)
                    ctx.V, ctx.scale, ctx.w_dtype = W.shape[0], scale, W.dtype
                    return embed(ids, W, scale)

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, g):
                    (ids,) = ctx.saved_tensors
                    dW = embed_bwd(ids, g.contiguous(), ctx.V, ctx.scale)
                    return None, dW.to(ctx.w_dtype), None

            cls._fn = Embedding
        return cls._fn


def embedding(ids, W, scale=1.0):
    """``embed`` as a differentiable torch function of W (gradient: ``embed_bwd``)."""
    return _Embedding.get().apply(ids, W, float(scale))


def _setting(torch, v, name, dtype, N, device):
    """(value, per-row array or None) of one sampling setting."""
    if not torch.is_tensor(v):
        return v, None
    if tuple(v.shape) != (N,) or v.dtype != dtype or v.device != device or not v.is_contiguous():
        raise ValueError(f"{name} must be a number or a contiguous {dtype} tensor [{N}] on {device}")
    return 0, v


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, ids_out=None, logp_out=None):
    """One token per row of logits [N, V] from the given random numbers u (float32 [N]
    in [0, 1)): (ids int32 [N], log-probabilities float32 [N]).

    Tokens are ordered by logit descending, equal logits by id ascending (as
    ``topk`` orders them) and weighed by exp(logit / temperature).  Kept is the
    shortest of: the first ``top_k`` (0: all), the shortest prefix with
    ``top_p`` of their mass, and the tokens at least ``min_p`` times as likely
    as the first.  The token is the first at which the kept tokens' cumulative
    probability exceeds u.  Each setting is a number or, for a batch of
    requests, a tensor [N] (float32; top_k int32).  Temperature 0 takes the
    largest logit.  Tokens at -inf or NaN are never drawn; a row without any
    other gives id -1 and log-probability -inf.

    logits are bfloat16 or float32 with adjacent elements in a row; rows may be
    strided (a slice of a padded vocabulary, the last position of a batch).
    """
    import torch

    dev = _gpu(logits, "logits")
    dt = _dtype(torch, logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [N, V]")
    N, V = logits.shape
    if V > 1 and N > 0 and logits.stride(1) != 1:
        raise ValueError("the elements of a row of logits must be adjacent")
    if u.dtype != torch.float32 or tuple(u.shape) != (N,) or u.device != dev or not u.is_contiguous():
        raise ValueError(f"u must be a contiguous float32 tensor [{N}] on {dev}")
    T, Ts = _setting(torch, temperature, "temperature", torch.float32, N, dev)
    k, ks = _setting(torch, top_k, "top_k", torch.int32, N, dev)
    p, ps = _setting(torch, top_p, "top_p", torch.float32, N, dev)
    m, ms = _setting(torch, min_p, "min_p", torch.float32, N, dev)
    how = Sampling(T, k, p, m, *(t.data_ptr() if t is not None else None for t in (Ts, ks, ps, ms)))
    _check_out(torch, ids_out, (N,), torch.int32, dev, "ids_out")
    _check_out(torch, logp_out, (N,), torch.float32, dev, "logp_out")
    if ids_out is None:
        ids_out = torch.empty((N,), dtype=torch.int32, device=dev)
    if logp_out is None:
        logp_out = torch.empty((N,), dtype=torch.float32, device=dev)
    with _on(torch, dev):
        _check(lib().ckl_sample(dt, _ptr(logits), N, V, logits.stride(0) if N > 1 else V, _ptr(u), ctypes.byref(how),
                                _ptr(ids_out), _ptr(logp_out), _stream(torch, dev)), "ckl_sample")
    return ids_out, logp_out
