"""Operators around the vocabulary table W [V, d], beside the loss at its head:
the embedding lookup and its gradient, sampling tokens from logits, and the
head's product with a weight held in 8 bits.

Argument checks and marshalling only, as in ``binding``: every step runs in the
library's HIP kernels on the current stream of the tensors' device, and CPU
tensors raise.
"""
from __future__ import annotations

import contextlib
import ctypes

from .binding import DTYPE_BF16, DTYPE_F32, Sampling, _check, _check_out, _ptr, lib, topk


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


def _stream(torch, device):
    """The current stream's handle.  torch's own short way to it spares a call on a
    few rows 2 of its 10 us; without it, through the Stream object."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw is not None else torch.cuda.current_stream(device).cuda_stream


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


def _not_capturing(torch, step):
    """autograd accumulates a leaf's gradient on the stream where its accumulator was
    made, which an eager graph of the same leaf may have left outside the capture:
    that would end the process, so it is refused first."""
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"embedding's {step} cannot be captured with a gradient: capture embed and embed_bwd")


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
                    _not_capturing(torch, "backward")
                    (ids,) = ctx.saved_tensors
                    dW = embed_bwd(ids, g.contiguous(), ctx.V, ctx.scale)
                    return None, dW.to(ctx.w_dtype), None

            cls._fn = Embedding
        return cls._fn


def embedding(ids, W, scale=1.0):
    """``embed`` as a differentiable torch function of W (gradient: ``embed_bwd``).

    W is copied where it is not contiguous, in every call; a bfloat16 W's gradient
    is summed in a float32 [V, d] and then rounded.  A stream capture takes it only
    where no gradient is asked for; a captured training step calls ``embed`` and
    ``embed_bwd``.
    """
    import torch

    if W.requires_grad and torch.is_grad_enabled():
        _not_capturing(torch, "forward")
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
    need = ctypes.c_uint64(0)
    _check(lib().ckl_sample_workspace(dt, N, V, ctypes.byref(need)), "ckl_sample_workspace")
    with _on(torch, dev):
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
        _check(lib().ckl_sample(dt, _ptr(logits), N, V, logits.stride(0) if N > 1 else V, _ptr(u), ctypes.byref(how),
                                _ptr(ids_out), _ptr(logp_out), _ptr(ws), need.value, _stream(torch, dev)), "ckl_sample")
    return ids_out, logp_out


def quantize_fp8(x, block_rows=1):
    """(q float8_e4m3fn [R, C], scales float32): x in 8 bits, an element being q times
    the scale of its block.

    ``block_rows`` = 1 (rows, activations): one scale per 1 x 128 block, scales
    [ceil(C / 128), R]; 128 (a weight): one per 128 x 128 block, scales
    [ceil(R / 128), ceil(C / 128)].  scale = amax / 448, q rounded to nearest
    even; values that are not finite become NaN.  x is bfloat16 or float32,
    contiguous, C a multiple of 16.
    """
    import torch

    dev = _gpu(x, "x")
    dt = _dtype(torch, x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [R, C] tensor")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    R, C = x.shape
    kb = -(-C // 128)
    q = torch.empty((R, C), dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.empty((kb, R) if block_rows == 1 else (-(-R // 128), kb), dtype=torch.float32, device=dev)
    with _on(torch, dev):
        _check(lib().ckl_quantize_fp8(dt, _ptr(x), R, C, block_rows, _ptr(q), _ptr(scales), _stream(torch, dev)),
               "ckl_quantize_fp8")
    return q, scales


def _check_fp8(torch, q, scales, shape, name, dev):
    if q.dtype != torch.float8_e4m3fn or q.dim() != 2 or not q.is_contiguous() or q.device != dev:
        raise ValueError(f"{name}q must be a contiguous 2-D float8_e4m3fn tensor on {dev}")
    _check_out(torch, scales, shape, torch.float32, dev, f"{name}s")


def matmul_fp8(xq, xs, wq, ws, dtype=None, out=None):
    """xq [M, d] times the transposed weight wq [V, d], both in 8 bits with the scales
    ``quantize_fp8`` gives (rows, and a weight): [M, V] in ``dtype`` (bfloat16 if
    None, or float32), summed in fp32 and rounded once.  For bfloat16 results,
    products 14 bits below the largest of their 8 may be dropped, except in calls
    of up to 16 rows under fewer than 16,384 ids, or of one or two rows under a
    weight of more than 2^28 values: there a row's results can differ from those
    that it has among more rows, within that bound.  No gradient."""
    import torch

    dev = _gpu(xq, "xq")
    if xq.dim() != 2 or wq.dim() != 2 or xq.shape[1] != wq.shape[1]:
        raise ValueError("xq must be [M, d] and wq [V, d]")
    (M, d), V = xq.shape, wq.shape[0]
    kb = -(-d // 128)
    _check_fp8(torch, xq, xs, (kb, M), "x", dev)
    _check_fp8(torch, wq, ws, (-(-V // 128), kb), "w", dev)
    if dtype is None:
        dtype = out.dtype if out is not None else torch.bfloat16
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be bfloat16 or float32")
    _check_out(torch, out, (M, V), dtype, dev, "out")
    if out is None:
        out = torch.empty((M, V), dtype=dtype, device=dev)
    dt = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32
    with _on(torch, dev):
        _check(lib().ckl_matmul_fp8(dt, _ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), M, V, d, _ptr(out),
                                    _stream(torch, dev)), "ckl_matmul_fp8")
    return out


def logits_fp8(H, wq, ws, dtype=None, out=None):
    """Logits [M, V] of hidden states H [M, d] (bfloat16 or float32) under a head held
    in 8 bits (``wq``, ``ws`` = ``quantize_fp8(W, 128)``, once): H's rows are
    quantised in the call, then ``matmul_fp8``, whose accuracy and results they
    have (``dtype`` float32 keeps every product).  No gradient."""
    xq, xs = quantize_fp8(H)
    return matmul_fp8(xq, xs, wq, ws, dtype=dtype, out=out)


def teacher_topk(H, wq, ws, K, chunk=0):
    """The teacher cache of hidden states H [N, d] under a head held in 8 bits: (ids
    int32 [N, K], values float32 [N, K]) as ``topk`` of their bfloat16 logits.

    Positions go in chunks (``chunk`` rows; 0: about 1 GiB of logits), so the
    N x V logits are never held at once.  The logits are ``logits_fp8`` of each
    chunk: with ``chunk`` 0 they are those of all rows in one call, a given chunk
    of few rows may take the product's other arithmetic (see ``matmul_fp8``).  As
    for ``topk``, NaN logits (a hidden row that is not finite) are outside its
    inputs.
    """
    import torch

    dev = _gpu(H, "H")
    if H.dim() != 2 or wq.dim() != 2:
        raise ValueError("H must be [N, d] and wq [V, d]")
    N, V, K, chunk = H.shape[0], wq.shape[0], int(K), int(chunk)
    if chunk < 0 or K < 1 or K > V:
        raise ValueError("chunk must be at least 0 and K in 1 .. V")
    least = 0  # rows of the last chunk: a few rows could take another kernel than the chunks before
    if chunk == 0:
        chunk = max(1, (1 << 30) // (2 * V))
        chunk = chunk // 256 * 256 or chunk
        least = min(128, chunk // 2)
    ids = torch.empty((N, K), dtype=torch.int32, device=dev)
    vals = torch.empty((N, K), dtype=torch.float32, device=dev)
    logits = torch.empty((min(chunk, N), V), dtype=torch.bfloat16, device=dev)
    with _on(torch, dev):
        r = 0
        while r < N:
            n = min(chunk, N - r)
            if 0 < N - r - n < least:
                n = N - r - least
            logits_fp8(H[r:r + n], wq, ws, out=logits[:n])
            topk(logits[:n], K, ids_out=ids[r:r + n], vals_out=vals[r:r + n])
            r += n
    return ids, vals
