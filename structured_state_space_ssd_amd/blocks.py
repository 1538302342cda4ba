"""The operators that make a recurrent block of a model: the gated linear
recurrence, the join of a block's output with the residual stream and its
norms, and dropout.

Like ``layers`` these check tensor metadata, allocate outputs and workspaces
with torch and call the C ABI (include/ssd.h); nothing here computes. Work is
enqueued on the current stream of the tensors' device. Activations may be
slices of a wider projection: their last axis has to be contiguous, the others
can have any stride. Parameters, states, gradients that come in and outputs
are dense.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native
from ._native import dtype_code
from .layers import _call, _f32, _int_sizes, _on_gpu, _param, _required, _rows, _slice, _workspace

__all__ = ["recurrence_forward", "recurrence_backward", "recurrence_step", "block_norm_forward",
           "block_norm_backward", "dropout"]

KEEP = 16  # tokens between the states that recurrence_forward keeps for recurrence_backward


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(x):
    """A new dense tensor like x (the shorter way where x is dense: 0.4 us of a token's call)."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


# ---- gated linear recurrence ------------------------------------------------------

def _recurrence_args(x, r, i, decay, z, ndim):
    """Checked addresses of the inputs and their strides."""
    _required(x=x, r=r)
    xs = x.shape
    if len(xs) != ndim:
        raise ValueError("x must be [Bt, E]" if ndim == 2 else "x must be [Bt, L, E]")
    _int_sizes(*xs)
    if (i is None) != (decay is None):
        raise ValueError("i and decay go together: both, or neither where r is the log-decay")
    dtype, device = x.dtype, x.get_device()
    pointers, strides = [], []  # strides: (batch, token)
    for t, name in ((x, "x"), (r, "r"), (i, "i"), (z, "z")):
        if t is None:
            pointers.append(None)
            strides += (0, 0)
            continue
        s = t.stride()
        # one test where all is well: a token's call makes four of these
        if t.shape == xs and t.dtype is dtype and s[-1] == 1 and t.get_device() == device:
            pointers.append(t.data_ptr())
        else:
            pointers.append(_slice(t, name, xs, x))
        strides += (s[0], s[1] if ndim == 3 else 0)
    pointers.insert(3, _param(decay, "decay", xs[-1:], x))
    return pointers, ctypes.byref(_native.SsdRecurrenceStrides(*strides))


def _recurrence_packed(cu_seqlens, x, init_state):
    if cu_seqlens is None:
        return None, 0
    if x.shape[0] != 1 or init_state is not None:
        raise ValueError("packed sequences use batch 1 and no init_state")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [nseq + 1]")
    _int_sizes(cu_seqlens.numel())
    return _param(cu_seqlens, "cu_seqlens", cu_seqlens.shape, x, torch.int32), cu_seqlens.numel() - 1


def recurrence_forward(x, r, i=None, decay=None, z=None, init_state=None, c=8.0, cu_seqlens=None,
                       return_final_state=False, return_states=False, workspace=None):
    """Gated linear recurrence with one state per channel over whole sequences
    (ssd_recurrence_forward): h_t = a_t h_{t-1} + u_t, y_t = h_t, or h_t silu(z_t) with z.

    With i and decay the gates are formed here, log a_t = -c softplus(decay)
    sigmoid(r_t) and u_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t; without them r is the
    log-decay itself, a_t = exp(r_t), and u_t = x_t. It is made for r at most 0: where r
    above 0 makes the decays of up to 256 tokens together pass float32, a state that is
    not zero becomes infinite or NaN there.
    x, r, i, z [Bt, L, E] float32 or bfloat16 (slices of wider projections are
    fine), decay [E] float32, init_state [Bt, E] float32 or None (zeros).
    cu_seqlens: packed sequences as for ``forward_varlen`` (Bt 1, no init_state);
    tokens in front of the first and behind the last one give zeros.
    Returns y, or a tuple of y, final_state ([Bt or nseq, E] float32, if
    requested) and states (if requested; float32, for recurrence_backward).
    """
    p, st = _recurrence_args(x, r, i, decay, z, 3)
    Bt, L, E = x.shape
    ip = _param(init_state, "init_state", (Bt, E), x)
    cp, nseq = _recurrence_packed(cu_seqlens, x, init_state)
    _on_gpu(x)
    code = dtype_code(x.dtype)
    y = _like(x)
    final = x.new_empty((nseq or Bt, E), dtype=_f32) if return_final_state else None
    states = x.new_empty((Bt, -(-L // KEEP), E), dtype=_f32) if return_states else None
    need = _native.lib.ssd_recurrence_forward_workspace_size(Bt, L, E, int(nseq > 0), code)
    keep, ws, ws_bytes = _workspace(workspace, need, x)
    _call(_native.lib.ssd_recurrence_forward, "ssd_recurrence_forward", x.device, *p[:4], c, p[4], Bt, L, E,
          code, ip, cp, nseq, y.data_ptr(), _ptr(final), _ptr(states), ws, ws_bytes, st)
    out = (y,) + ((final,) if return_final_state else ()) + ((states,) if return_states else ())
    return out if len(out) > 1 else y


def recurrence_backward(x, r, i, decay, dy, z=None, init_state=None, dfinal_state=None, c=8.0,
                        cu_seqlens=None, states=None, workspace=None):
    """Gradients of sum(dy * y) + sum(dfinal_state * final_state) for
    ``recurrence_forward`` with the same inputs (ssd_recurrence_backward).

    states: what recurrence_forward returned of that name for the same inputs;
    None: they are made again, at the cost of reading x, r, i and z once more.
    dfinal_state: like final_state ([nseq, E] with cu_seqlens).
    Returns a dict: dx, dr, di, dz (dense, in x's type), ddecay [E] and dinit
    [Bt, E] float32; di and ddecay are None without decay, dz without z, dinit
    without init_state.
    """
    p, st = _recurrence_args(x, r, i, decay, z, 3)
    _required(dy=dy)
    Bt, L, E = x.shape
    yp = _param(dy, "dy", x.shape, x, x.dtype)
    ip = _param(init_state, "init_state", (Bt, E), x)
    cp, nseq = _recurrence_packed(cu_seqlens, x, init_state)
    fp = _param(dfinal_state, "dfinal_state", (nseq or Bt, E), x)
    sp = _param(states, "states", (Bt, -(-L // KEEP), E), x)
    _on_gpu(x)
    code = dtype_code(x.dtype)
    new = lambda on, shape=(Bt, L, E), dtype=x.dtype: x.new_empty(shape, dtype=dtype) if on else None  # noqa: E731
    gated = decay is not None
    out = {"dx": new(True), "dr": new(True), "di": new(gated), "ddecay": new(gated, (E,), _f32),
           "dz": new(z is not None), "dinit": new(init_state is not None, (Bt, E), _f32)}
    need = _native.lib.ssd_recurrence_backward_workspace_size(Bt, L, E, int(nseq > 0), int(states is not None), code)
    keep, ws, ws_bytes = _workspace(workspace, need, x)
    _call(_native.lib.ssd_recurrence_backward, "ssd_recurrence_backward", x.device, *p[:4], c, p[4], ip, cp,
          nseq, sp, yp, fp, Bt, L, E, code, *map(_ptr, out.values()), ws, ws_bytes, st)
    return out


def recurrence_step(state, x, r, i=None, decay=None, z=None, c=8.0):
    """One token of ``recurrence_forward`` for every sequence (ssd_recurrence_step):
    x, r, i, z [Bt, E]; ``state`` [Bt, E] float32, recurrence_forward's
    final_state at first, is updated in place. Returns y [Bt, E].
    """
    p, st = _recurrence_args(x, r, i, decay, z, 2)
    _required(state=state)
    Bt, E = x.shape
    sp = _param(state, "state", (Bt, E), x)
    _on_gpu(x)
    y = _like(x)
    _call(_native.lib.ssd_recurrence_step, "ssd_recurrence_step", x.device, sp, *p[:4], c, p[4], Bt, E,
          dtype_code(x.dtype), y.data_ptr(), st)
    return y


# ---- dropout ------------------------------------------------------------------------

def _random(p, rng, like):
    """ssd_random of the share p and (seed, offset), or None where nothing is dropped."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be between 0 and 1, got {p}")
    if rng is None:
        if p:
            raise ValueError("rng is required: (seed, offset), or an int64 tensor of the two")
        return None
    if isinstance(rng, torch.Tensor):
        return ctypes.byref(_native.SsdRandom(p, 0, 0, _param(rng, "rng", (2,), like, torch.int64)))
    seed, offset = rng
    if not (isinstance(seed, int) and isinstance(offset, int)):
        raise TypeError("rng must be two integers or an int64 tensor")
    return ctypes.byref(_native.SsdRandom(p, seed & 0xffffffffffffffff, offset & 0xffffffffffffffff, None))


def dropout(x, p, rng):
    """x / (1 - p) where an element stays, 0 where it is dropped (ssd_dropout); the mask is
    computed from rng and the element's place and never stored. The same call on the
    gradient is the backward pass.

    x [..., D] float32 or bfloat16, rows evenly spaced (a slice of a wider tensor is
    fine). p: the share that is dropped, taken to the nearest 1/65536. rng: (seed,
    offset) as integers, or an int64 tensor of the two on x's device, which a captured
    graph reads at every replay; the same pair drops the same elements of [rows, D].
    """
    _required(x=x)
    rows, step = _rows(x, "x")
    rp = _random(p, (0, 0) if rng is None and not p else rng, x)
    _on_gpu(x)
    code = dtype_code(x.dtype)
    y = _like(x)
    _call(_native.lib.ssd_dropout, "ssd_dropout", x.device, x.data_ptr(), step, rows, x.shape[-1], rp, code,
          y.data_ptr())
    return y


# ---- block norm ---------------------------------------------------------------------

def _block(x, weight, bias, post_weight, post_bias, scale, residual_scale, branch_scale, rms, eps):
    D = x.shape[-1:]
    if weight is None and post_weight is None:
        raise ValueError("weight or post_weight is required")
    for w, b, name in ((weight, bias, "bias"), (post_weight, post_bias, "post_bias")):
        if w is None and b is not None:
            raise ValueError(f"{name} without its weight")
    return ctypes.byref(_native.SsdBlock(
        _param(weight, "weight", D, x), _param(bias, "bias", D, x), _param(post_weight, "post_weight", D, x),
        _param(post_bias, "post_bias", D, x), _param(scale, "scale", D, x), residual_scale, branch_scale,
        int(bool(rms)), eps))


def _stream_code(stream, name, x):
    if stream.dtype != _f32 and stream.dtype != x.dtype:
        raise TypeError(f"{name} must be float32 or {x.dtype}, got {stream.dtype}")
    return dtype_code(stream.dtype)


def block_norm_forward(x, residual, weight=None, bias=None, post_weight=None, post_bias=None, scale=None,
                       z=None, residual_scale=1.0, branch_scale=1.0, p=0.0, rng=None, eps=1e-5, rms=False,
                       return_stats=False):
    """A block's output joined with the residual stream, and the next block's input
    (ssd_block_norm_forward):
    sum = residual_scale * residual + branch_scale * dropout(norm(x) * scale * silu(z)),
    y = norm(sum). Where that is only residual + x and its norm, ``norm_forward`` with a
    residual does the same, and its backward reads less.

    post_weight, post_bias: of the norm after the block (of x; None: x itself);
    weight, bias: of the norm before the next (None: no y). Layer norms, with rms their
    root-mean-square form. scale [D]: a factor per column; z like x: a gate per
    element; p, rng: see ``dropout``. Each may be left out, but not both norms.
    x [..., D] float32 or bfloat16, D at most 8192, rows evenly spaced; residual like
    x, in x's type or float32; weights, biases and scale [D] float32.
    Returns (y, sum), sum in residual's type, and with return_stats the statistics
    that block_norm_backward takes.
    """
    _required(x=x, residual=residual)
    rows, step = _rows(x, "x")
    block = _block(x, weight, bias, post_weight, post_bias, scale, residual_scale, branch_scale, rms, eps)
    rcode = _stream_code(residual, "residual", x)
    rp = _param(residual, "residual", x.shape, x, residual.dtype)
    zp = _slice(z, "z", x.shape, x)
    zstep = 0 if z is None else _rows(z, "z")[1]
    random = _random(p, rng, x)
    _on_gpu(x)
    code = dtype_code(x.dtype)
    total = torch.empty_like(residual)
    y = None if weight is None else _like(x)
    stats = (None,) * 4
    if return_stats:
        new = lambda on: x.new_empty(x.shape[:-1], dtype=_f32) if on else None  # noqa: E731
        pre, post = weight is not None, post_weight is not None
        stats = (new(pre and not rms), new(pre), new(post and not rms), new(post))
    _call(_native.lib.ssd_block_norm_forward, "ssd_block_norm_forward", x.device, x.data_ptr(), step, rp, rcode,
          zp, zstep, block, random, rows, x.shape[-1], code, _ptr(y), total.data_ptr(), *map(_ptr, stats))
    return (y, total, stats) if return_stats else (y, total)


def block_norm_backward(dy, dsum, x, total, stats, weight=None, bias=None, post_weight=None, post_bias=None,
                        scale=None, z=None, residual_scale=1.0, branch_scale=1.0, p=0.0, rng=None,
                        workspace=None):
    """Gradients of ``block_norm_forward`` (ssd_block_norm_backward), given the same
    arguments.

    dy: the gradient of y (None where there was none); dsum: of sum, by the ways that do
    not go through y (None: none). total, stats: the sum and the statistics that
    block_norm_forward returned.
    Returns a dict: dx and dz (x's type), dresidual (total's type), dweight, dbias,
    dpost_weight, dpost_bias and dscale ([D] float32), None where their tensor was.
    """
    _required(x=x, total=total, stats=stats)
    rows, step = _rows(x, "x")
    mean, rstd, post_mean, post_rstd = stats
    rms = mean is None and post_mean is None
    block = _block(x, weight, bias, post_weight, post_bias, scale, residual_scale, branch_scale, rms, 0.0)
    tcode = _stream_code(total, "total", x)
    tp = _param(total, "total", x.shape, x, total.dtype)
    if (dy is None) != (weight is None):
        raise ValueError("dy goes with weight")
    dyp = _param(dy, "dy", x.shape, x, x.dtype)
    dsp = _param(dsum, "dsum", x.shape, x, total.dtype)
    if weight is not None:
        _required(rstd=rstd)
    if post_weight is not None:
        _required(post_rstd=post_rstd)
    sp = [_param(t, name, x.shape[:-1], x) for t, name in
          ((mean, "mean"), (rstd, "rstd"), (post_mean, "post_mean"), (post_rstd, "post_rstd"))]
    zp = _slice(z, "z", x.shape, x)
    zstep = 0 if z is None else _rows(z, "z")[1]
    random = _random(p, rng, x)
    _on_gpu(x)
    code = dtype_code(x.dtype)
    like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    out = {"dx": _like(x), "dresidual": torch.empty_like(total), "dz": None if z is None else _like(x),
           "dweight": like(weight), "dbias": like(bias), "dpost_weight": like(post_weight),
           "dpost_bias": like(post_bias), "dscale": like(scale)}
    need = _native.lib.ssd_block_norm_backward_workspace_size(rows, x.shape[-1], code)
    keep, ws, ws_bytes = _workspace(workspace, need, x)
    _call(_native.lib.ssd_block_norm_backward, "ssd_block_norm_backward", x.device, dyp, dsp, x.data_ptr(), step,
          tp, tcode, zp, zstep, block, random, *sp, rows, x.shape[-1], code, *map(_ptr, out.values()), ws,
          ws_bytes)
    return out
