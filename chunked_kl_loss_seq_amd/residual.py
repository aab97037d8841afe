"""The end of a block, up to the hidden states that the loss takes: the residual's
norms before and after it, with gate, scale and dropout, and dropout on its own.

Argument checks and marshalling only, as in ``binding``: every step runs in the
library's HIP kernels on the current stream of the tensors' device, and CPU
tensors raise.
"""
from __future__ import annotations

import ctypes

from .binding import Drop, Norm, _check, _check_out, lib
from .vocab import _dtype, _gpu, _stream


def _at(t):
    """Address of a tensor, or None."""
    return None if t is None else t.data_ptr()


def _call(torch, device, fn, *args):
    """fn(*args, the device's current stream), on that device: the library launches on
    the current one."""
    if torch.cuda.current_device() == device.index:
        st = fn(*args, _stream(torch, device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _stream(torch, device))
    if st:
        _check(st, fn.__name__)


_WORD = (1 << 64) - 1


def _drop(torch, p, seed, offset, device):
    """The fields of ckl_drop for a probability, a seed in [0, 2^64) and an offset: an int
    in [0, 2^64) or an int64 GPU tensor of one element, read when the kernels run."""
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in [0, 1]")
    if not 0 <= seed <= _WORD:
        raise ValueError("seed must be in [0, 2^64)")
    if isinstance(offset, torch.Tensor):
        if offset.dtype != torch.int64 or offset.numel() != 1 or offset.device != device:
            raise ValueError(f"offset must be an int or an int64 tensor of one element on {device}")
        return p, seed, 0, offset.data_ptr()
    if not 0 <= offset <= _WORD:
        raise ValueError("offset must be in [0, 2^64)")
    return p, seed, offset, None


def drop(x, p, seed, offset=0, out=None):
    """x with elements set to zero with probability ``p`` and the others divided by
    1 - p, in fp32, rounded once.  x: bfloat16 or float32, contiguous, any shape.

    The mask follows from (seed, offset, element index) by a counter-based
    generator and is never stored: the gradient is the same call on the upstream
    gradient.  ``p`` counts in steps of 2^-16, and what is kept is divided by 1
    minus the rounded p.  ``offset`` is an int or an int64 GPU tensor of one
    element, read when the kernel runs: a captured step that adds to it draws
    another mask in every replay (its gradient has to run before the addition).
    ``out`` may be x.
    """
    import torch

    dev = _gpu(x, "x")
    dt = _dtype(torch, x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    how = Drop(*_drop(torch, p, seed, offset, dev))
    if out is None:
        out = torch.empty_like(x)
    else:
        _check_out(torch, out, x.shape, x.dtype, dev, "out")
    _call(torch, dev, lib().ckl_dropout, dt, x.data_ptr(), x.numel(), how, out.data_ptr())
    return out


def _no_capture(torch, what, use):
    """autograd accumulates a leaf's gradient on the stream where its accumulator was
    made, which an eager graph of the same leaf may have left outside the capture:
    that would end the process, so it is refused first."""
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{what} cannot be captured with a gradient: capture {use}")


class _Dropout:
    """torch.autograd.Function wrapper, created lazily so importing needs no torch."""

    _fn = None

    @classmethod
    def get(cls):
        if cls._fn is None:
            import torch

            class Dropout(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x, p, seed, offset):
                    ctx.how = (p, seed)
                    # a copy of a device offset: the caller may move it on before the gradient
                    ctx.offset = offset.clone() if torch.is_tensor(offset) else offset
                    return drop(x.contiguous(), p, seed, ctx.offset)

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, g):
                    _no_capture(torch, "dropout's backward", "drop")
                    return drop(g.contiguous(), *ctx.how, ctx.offset), None, None, None

            cls._fn = Dropout
        return cls._fn


def dropout(x, p, seed, offset=0):
    """``drop`` as a differentiable torch function of x, which is copied where it is not
    contiguous.  A stream capture takes it only where no gradient is asked for; a
    captured training step calls ``drop`` in both directions."""
    import torch

    if x.requires_grad and torch.is_grad_enabled():
        _no_capture(torch, "dropout's forward", "drop")
        return _Dropout.get().apply(x, p, seed, offset)
    return drop(x.contiguous(), p, seed, offset)


def _norm_args(torch, y, r, w_pre, w_post, gate, scale, p, seed, offset, eps):
    """Checks what both directions share: (dtype code, device, N, d, ckl_norm)."""
    dev = _gpu(y, "y")
    dt, kind, shape = _dtype(torch, y, "y"), y.dtype, y.shape
    if y.dim() < 1 or shape[-1] == 0:
        raise ValueError("y must be [..., d], d at least 1")
    if r.shape != shape:
        raise ValueError("r must have the shape of y")
    d = shape[-1]
    for name, t in (("y", y), ("r", r), ("w_pre", w_pre), ("w_post", w_post), ("gate", gate)):
        if t is not None and (t.dtype != kind or t.device != dev or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {kind} tensor on {dev}")
    if w_pre is not None and (w_pre.dim() != 1 or w_pre.shape[0] != d):
        raise ValueError(f"w_pre must be [{d}]")
    if w_post is not None and (w_post.dim() != 1 or w_post.shape[0] != d):
        raise ValueError(f"w_post must be [{d}]")
    rows = False
    if gate is not None and (gate.dim() != 1 or gate.shape[0] != d):
        if gate.shape != shape:
            raise ValueError(f"gate must be [{d}] or have the shape of y")
        rows = True
    eps = float(eps)
    if not eps >= 0.0:
        raise ValueError("eps must be at least 0")
    drops = _drop(torch, p, seed, offset, dev)
    how = Norm(_at(w_post), _at(w_pre), _at(gate), 1 if rows else 0, scale, eps,
               ctypes.pointer(Drop(*drops)) if p else None)
    return dt, dev, y.numel() // d, d, how


def add_norm(y, r, w_pre, w_post=None, gate=None, scale=1.0, p=0.0, seed=0, offset=0, eps=1e-6, stats=False,
             r_out=None, x_out=None):
    """The residual's norms around a block: (r_out, x, stats).

    With rms(v) = sqrt(mean(v^2) + eps) over the last dimension,
      u     = w_post y / rms(y)          (u = y without ``w_post``)
      r_out = r + scale gate drop(u)     (``drop`` with p, seed, offset; gate [d], of y's shape, or None)
      x     = w_pre r_out / rms(r_out)   (None without ``w_pre``)
    in fp32, r_out and x each rounded once to the inputs' type (x from the fp32
    r_out).  y and r [..., d] and the weights are all bfloat16 or all float32,
    contiguous; d a multiple of 8, at most 16,384.  After the last block, x is the
    H of the loss.

    ``stats`` = True keeps the rows' float32 reciprocal rms [2, N] for
    ``add_norm_bwd``; otherwise it is None.  ``r_out`` may be r where no gradient
    is needed.
    """
    import torch

    dt, dev, N, d, how = _norm_args(torch, y, r, w_pre, w_post, gate, scale, p, seed, offset, eps)
    if r_out is None:
        r_out = torch.empty_like(y)
    else:
        _check_out(torch, r_out, y.shape, y.dtype, dev, "r_out")
    if x_out is not None:
        if w_pre is None:
            raise ValueError("x_out needs w_pre")
        _check_out(torch, x_out, y.shape, y.dtype, dev, "x_out")
    elif w_pre is not None:
        x_out = torch.empty_like(y)
    kept = torch.empty((2, N), dtype=torch.float32, device=dev) if stats else None
    _call(torch, dev, lib().ckl_add_norm, dt, y.data_ptr(), r.data_ptr(), how, N, d, r_out.data_ptr(), _at(x_out),
          _at(kept))
    return r_out, x_out, kept


def add_norm_bwd(y, r, w_pre, w_post, stats, dx, dr_out, gate=None, scale=1.0, p=0.0, seed=0, offset=0, eps=1e-6):
    """Gradients of ``add_norm``: (dy, dr, dw_post, dw_pre, dgate), None where there is
    no such input.

    y, r, the weights and settings are the forward call's, ``stats`` its reciprocal
    rms; dx and dr_out are the gradients of x and r_out (either may be None, not
    both).  dy, dr and the gradient of a gate of y's shape have y's type; dw_post,
    dw_pre and the gradient of a gate [d] are float32, summed in a fixed order.
    """
    import torch

    dt, dev, N, d, how = _norm_args(torch, y, r, w_pre, w_post, gate, scale, p, seed, offset, eps)
    _check_out(torch, stats, (2, N), torch.float32, dev, "stats")
    _check_out(torch, dx, y.shape, y.dtype, dev, "dx")
    _check_out(torch, dr_out, y.shape, y.dtype, dev, "dr_out")
    if stats is None:
        raise ValueError("add_norm_bwd needs the stats of add_norm(..., stats=True)")
    if dx is None and dr_out is None:
        raise ValueError("dx or dr_out must be given")
    if dx is not None and w_pre is None:
        raise ValueError("dx needs w_pre")
    dy, dr = torch.empty_like(y), torch.empty_like(y)
    vec = lambda: torch.empty((d,), dtype=torch.float32, device=dev)  # noqa: E731
    dw_post = vec() if w_post is not None else None
    dw_pre = vec() if w_pre is not None else None
    dgate = None if gate is None else torch.empty_like(gate) if how.gate_rows else vec()
    sums = (w_post is not None) + (w_pre is not None) + (gate is not None and not how.gate_rows)
    need = ctypes.c_uint64(0)
    _check(lib().ckl_add_norm_bwd_workspace(N, d, sums, need), "ckl_add_norm_bwd_workspace")
    # from torch's allocator, so that calls on several streams, or captured into several graphs, never share it
    ws = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
    _call(torch, dev, lib().ckl_add_norm_bwd, dt, y.data_ptr(), r.data_ptr(), how, N, d, stats.data_ptr(), _at(dx),
          _at(dr_out), dy.data_ptr(), dr.data_ptr(), _at(dw_post), _at(dw_pre), _at(dgate), _at(ws), need.value)
    return dy, dr, dw_post, dw_pre, dgate


class _ResidualNorm:
    """torch.autograd.Function wrapper, created lazily so importing needs no torch."""

    _fn = None

    @classmethod
    def get(cls):
        if cls._fn is None:
            import torch

            class ResidualNorm(torch.autograd.Function):
                @staticmethod
                def forward(ctx, y, r, w_pre, w_post, gate, scale, p, seed, offset, eps):
                    y, r, w_pre, w_post, gate = (None if t is None else t.contiguous()
                                                 for t in (y, r, w_pre, w_post, gate))
                    ctx.set_materialize_grads(False)
                    offset = offset.clone() if torch.is_tensor(offset) else offset
                    ctx.how = {"scale": scale, "p": p, "seed": seed, "offset": offset, "eps": eps}
                    r_out, x, stats = add_norm(y, r, w_pre, w_post, gate, stats=True, **ctx.how)
                    ctx.save_for_backward(y, r, w_pre, w_post, gate, stats)
                    return r_out, x

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, dr_out, dx):
                    _no_capture(torch, "residual_norm's backward", "add_norm and add_norm_bwd")
                    y, r, w_pre, w_post, gate, stats = ctx.saved_tensors
                    if dr_out is None and dx is None:
                        return (None,) * 10
                    dr_out, dx = (None if g is None else g.contiguous() for g in (dr_out, dx))
                    dy, dr, dw_post, dw_pre, dgate = add_norm_bwd(y, r, w_pre, w_post, stats, dx, dr_out, gate, **ctx.how)
                    cast = lambda g, t: None if g is None else g.to(t.dtype)  # noqa: E731
                    return (dy, dr, cast(dw_pre, w_pre), cast(dw_post, w_post), cast(dgate, gate), None, None, None, None,
                            None)

            cls._fn = ResidualNorm
        return cls._fn


def residual_norm(y, r, w_pre, w_post=None, gate=None, scale=1.0, p=0.0, seed=0, offset=0, eps=1e-6):
    """``add_norm`` as a differentiable torch function of y, r, the weights and the gate:
    (r_out, x).  Inputs are copied where they are not contiguous.  A stream capture
    takes it only where no gradient is asked for; a captured training step calls
    ``add_norm`` and ``add_norm_bwd``."""
    import torch

    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (y, r, w_pre, w_post, gate)):
        _no_capture(torch, "residual_norm's forward", "add_norm and add_norm_bwd")
    return _ResidualNorm.get().apply(y, r, w_pre, w_post, gate, scale, p, seed, offset, eps)
