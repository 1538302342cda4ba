"""The operators around the state-space layer: the short causal convolution,
the selective scan and the normalisation.

Like the package's other functions these check tensor metadata, allocate
outputs and workspaces with torch and call the C ABI (include/ssd.h); nothing
here computes. Work is enqueued on the current stream of the tensors' device.
Activations may be slices of a wider projection: their last axis has to be
contiguous, the others can have any stride. Parameters, states, gradients that
come in and outputs are dense.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native
from ._native import check, dtype_code

__all__ = ["conv_forward", "conv_backward", "conv_step", "selective_forward", "selective_backward",
           "selective_step", "norm_forward", "norm_backward"]

_f32 = torch.float32


def _param(t, name, shape, like, dtype=_f32):
    """Address of a dense tensor of this shape and type next to `like` (None: NULL)."""
    if t is None:
        return None
    # one test where all is well: a token's call makes up to a dozen of these
    if (t.shape == shape and t.dtype is dtype and t.is_contiguous()
            and t.get_device() == like.get_device()):
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, x on {like.device}")


def _slice(t, name, shape, like):
    """Address of an activation of this shape and like's type whose last axis is contiguous."""
    if t is None:
        return None
    if (t.shape == shape and t.dtype is like.dtype and (t.stride(-1) == 1 or t.shape[-1] == 1)
            and t.get_device() == like.get_device()):
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    raise ValueError(f"{name} is on {t.device}, x on {like.device}")


def _required(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} is required")


def _int_sizes(*sizes):
    # the C ABI's sizes are ints, of which ctypes would pass the low 32 bits
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"sizes must be below 2^31, got {sizes}")


def _on_gpu(x):
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")


def _call(fn, where, device, *args):
    """fn(*args, the device's current stream), with that device the current one."""
    # The handle alone: torch.cuda.current_stream builds an object around it, 1.9 us
    # of a single token's 15 to 17.
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    check(rc, where)


def _workspace(workspace, need, x):
    """(address, bytes) of the caller's workspace, or of a new one of `need` bytes."""
    if workspace is None:
        workspace = x.new_empty(max(need, 1), dtype=torch.uint8)
    elif not workspace.is_contiguous() or workspace.device != x.device:
        raise ValueError("workspace must be a contiguous tensor on x's device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---- short causal convolution ---------------------------------------------------

def _conv_sizes(x, weight, ndim):
    _required(x=x, weight=weight)
    xs, ws = x.shape, weight.shape
    if len(xs) != ndim or len(ws) != 2 or ws[0] != xs[-1]:
        raise ValueError("x must be [Bt, K] and weight [K, W]" if ndim == 2 else
                         "x must be [Bt, L, K] and weight [K, W]")
    _int_sizes(*xs, ws[1])
    return ws[1]


def _conv_parts(split, K):
    """(ctypes int array or None, its length) of the channel split."""
    if split is None:
        return None, 0, (K,)
    split = tuple(int(k) for k in split)
    if not 1 <= len(split) <= 3 or min(split) < 1 or sum(split) != K:
        raise ValueError(f"split must be 1 to 3 positive sizes with sum {K}, got {split}")
    return (ctypes.c_int * len(split))(*split), len(split), split


_POINTERS = [ctypes.c_void_p * n for n in range(4)]


def _pointers(addresses):
    return _POINTERS[len(addresses)](*addresses)


def conv_forward(x, weight, bias=None, silu=True, init_state=None, return_final_state=False,
                 cu_seqlens=None, split=None):
    """y_t = act(bias + sum_k weight[:, k] x_{t-W+1+k}) over whole sequences
    (ssd_conv_forward): the causal convolution in front of the state-space layer.

    x [Bt, L, K] float32 or bfloat16 (a slice of a wider projection is fine),
    weight [K, W] with W = 2, 3 or 4 and bias [K] float32; act is SiLU or, with
    silu=False, nothing. init_state [Bt, W-1, K] in x's type: the inputs before
    the first token (None: zeros). cu_seqlens: packed sequences as for
    ``forward_varlen`` (Bt 1, no init_state). split: up to 3 sizes that cut the
    channels, e.g. (H * P, G * N, G * N); y is then a tuple of dense tensors,
    ready to be viewed as the layer's x, B and C.
    Returns y, or (y, final_state [Bt or nseq, W-1, K]) if requested.
    """
    W = _conv_sizes(x, weight, 3)
    Bt, L, K = x.shape
    arr, n, sizes = _conv_parts(split, K)
    xp = _slice(x, "x", x.shape, x)
    wp = _param(weight, "weight", (K, W), x)
    bp = _param(bias, "bias", (K,), x)
    ip = _param(init_state, "init_state", (Bt, W - 1, K), x, x.dtype)
    nseq, cp = 0, None
    if cu_seqlens is not None:
        if Bt != 1 or init_state is not None:
            raise ValueError("packed sequences use batch 1 and no init_state")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [nseq + 1]")
        _int_sizes(cu_seqlens.numel())
        nseq = cu_seqlens.numel() - 1
        cp = _param(cu_seqlens, "cu_seqlens", (nseq + 1,), x, torch.int32)
    _on_gpu(x)
    code = dtype_code(x.dtype)
    ys = [x.new_empty((Bt, L, k)) for k in sizes]
    final = None
    if return_final_state:
        final = x.new_empty((nseq or Bt, W - 1, K))
    _call(_native.lib.ssd_conv_forward, "ssd_conv_forward", x.device, xp, x.stride(0), x.stride(1),
          wp, bp, ip, cp, nseq, Bt, L, K, W, int(silu), code, arr, n,
          _pointers([y.data_ptr() for y in ys]), final.data_ptr() if final is not None else None)
    y = ys[0] if split is None else tuple(ys)
    return (y, final) if return_final_state else y


def conv_backward(x, weight, bias, dy, silu=True, init_state=None, dfinal_state=None,
                  workspace=None):
    """Gradients of sum(dy * y) + sum(dfinal_state * final_state) for
    ``conv_forward`` without cu_seqlens on the same inputs (ssd_conv_backward).

    dy: a tensor [Bt, L, K], or a sequence of up to 3 tensors that split the
    channels as conv_forward's y was. Returns a dict: dx [Bt, L, K] (x's type),
    dweight [K, W] float32, dbias ([K] float32, None without a bias) and dinit
    ([Bt, W-1, K] in x's type, None without an init_state).
    """
    W = _conv_sizes(x, weight, 3)
    _required(dy=dy)
    Bt, L, K = x.shape
    dys = [dy] if isinstance(dy, torch.Tensor) else list(dy)
    for d in dys:
        _required(dy=d)
    arr, n, sizes = _conv_parts([d.shape[-1] for d in dys], K)
    xp = _slice(x, "x", x.shape, x)
    wp = _param(weight, "weight", (K, W), x)
    bp = _param(bias, "bias", (K,), x)
    ip = _param(init_state, "init_state", (Bt, W - 1, K), x, x.dtype)
    fp = _param(dfinal_state, "dfinal_state", (Bt, W - 1, K), x, x.dtype)
    dp = [_param(d, "dy", (Bt, L, k), x, x.dtype) for d, k in zip(dys, sizes)]
    _on_gpu(x)
    code = dtype_code(x.dtype)
    out = {"dx": x.new_empty((Bt, L, K)),
           "dweight": torch.empty_like(weight),
           "dbias": None if bias is None else torch.empty_like(bias),
           "dinit": None if init_state is None else torch.empty_like(init_state)}
    need = _native.lib.ssd_conv_backward_workspace_size(Bt, L, K, W, code)
    keep, ws, ws_bytes = _workspace(workspace, need, x)
    _call(_native.lib.ssd_conv_backward, "ssd_conv_backward", x.device, xp, x.stride(0),
          x.stride(1), wp, bp, ip, arr, n, _pointers(dp), fp, Bt, L, K, W, int(silu), code,
          out["dx"].data_ptr(), out["dweight"].data_ptr(),
          None if bias is None else out["dbias"].data_ptr(),
          None if init_state is None else out["dinit"].data_ptr(), ws, ws_bytes)
    return out


def conv_step(state, x, weight, bias=None, silu=True, split=None):
    """One token of ``conv_forward`` for every sequence (ssd_conv_step): x [Bt, K];
    ``state`` [Bt, W-1, K] in x's type, conv_forward's final_state at first, is
    updated in place. Returns y [Bt, K], or the tuple of its parts with ``split``.
    """
    W = _conv_sizes(x, weight, 2)
    _required(state=state)
    Bt, K = x.shape
    arr, n, sizes = _conv_parts(split, K)
    xp = _slice(x, "x", x.shape, x)
    wp = _param(weight, "weight", (K, W), x)
    bp = _param(bias, "bias", (K,), x)
    sp = _param(state, "state", (Bt, W - 1, K), x, x.dtype)
    _on_gpu(x)
    ys = [x.new_empty((Bt, k)) for k in sizes]
    _call(_native.lib.ssd_conv_step, "ssd_conv_step", x.device, sp, xp, x.stride(0), wp, bp, Bt, K,
          W, int(silu), dtype_code(x.dtype), arr, n, _pointers([y.data_ptr() for y in ys]))
    return ys[0] if split is None else tuple(ys)


# ---- selective scan --------------------------------------------------------------

def _selective_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit):
    """Checked addresses of the scan's inputs, strides and options, and (G, N)."""
    _required(x=x, dt=dt, A=A, B=B, C=C)
    xs, bs = x.shape, B.shape
    lead = len(xs) - 1
    if lead not in (1, 2) or A.dim() != 2 or len(bs) != lead + 2 or bs[:lead] != xs[:lead]:
        raise ValueError("x must be [Bt, L, E], A [E, N] and B [Bt, L, G, N] (without L for one token)")
    E = xs[-1]
    G, N = bs[-2:]
    _int_sizes(*xs, G, N)
    if G < 1 or E % G:
        raise ValueError(f"{E} channels do not divide into {G} groups")
    pointers = [_slice(x, "x", xs, x), _slice(dt, "dt", xs, x), _param(A, "A", (E, N), x),
                _slice(B, "B", bs, x), _slice(C, "C", bs, x), _param(D, "D", (E,), x),
                _slice(z, "z", xs, x)]
    if G > 1:
        for t, name in ((B, "B"), (C, "C")):
            if t.stride(-2) != N:
                raise ValueError(f"{name}'s groups must be contiguous")
    strides = []  # (batch, token) of x, dt, z, B, C
    for t in (x, dt, z, B, C):
        s = (0, 0) if t is None else t.stride()
        strides += (s[0], s[1] if lead == 2 else 0)
    st = _native.SsdSelectiveStrides(*strides)
    opts = None
    if dt_bias is not None or dt_softplus or dt_limit is not None:
        lo, hi = (0.0, 0.0) if dt_limit is None else (float(dt_limit[0]), float(dt_limit[1]))
        opts = ctypes.byref(_native.SsdOptions(_param(dt_bias, "dt_bias", (E,), x),
                                               int(bool(dt_softplus)), int(dt_limit is not None),
                                               lo, hi, _native.SSD_DISC_EULER))
    return pointers, ctypes.byref(st), opts, G, N


def selective_forward(x, dt, A, B, C, D=None, z=None, init_state=None, return_final_state=False,
                      workspace=None, dt_bias=None, dt_softplus=False, dt_limit=None):
    """Selective scan with a decay rate per channel and state over whole
    sequences (ssd_selective_forward):
    h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t, y_t = (C_t h_t + D x_t) silu(z_t).

    x, dt, z (None: no gate) [Bt, L, E], B, C [Bt, L, G, N] (float32 or
    bfloat16, slices of wider projections are fine), A [E, N] and D [E] float32,
    init_state [Bt, E, N] float32 or None, N at most 64. dt_bias ([E]),
    dt_softplus, dt_limit: see ``options``.
    Returns y, or (y, final_state [Bt, E, N] float32) if requested.
    """
    p, st, opts, G, N = _selective_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    if x.dim() != 3:
        raise ValueError("x must be [Bt, L, E]")
    Bt, L, E = x.shape
    ip = _param(init_state, "init_state", (Bt, E, N), x)
    _on_gpu(x)
    code = dtype_code(x.dtype)
    y = x.new_empty((Bt, L, E))
    final = x.new_empty((Bt, E, N), dtype=_f32) if return_final_state else None
    need = _native.lib.ssd_selective_forward_workspace_size(Bt, L, E, G, N, code)
    keep, ws, ws_bytes = _workspace(workspace, need, x)
    _call(_native.lib.ssd_selective_forward, "ssd_selective_forward", x.device, *p, Bt, L, E, G, N,
          code, ip, y.data_ptr(), None if final is None else final.data_ptr(), ws, ws_bytes, st, opts)
    return (y, final) if return_final_state else y


def selective_backward(x, dt, A, B, C, D, dy, z=None, init_state=None, dfinal_state=None,
                       dt_bias=None, dt_softplus=False, dt_limit=None, workspace=None,
                       want_dinit=True):
    """Gradients of sum(dy * y) + sum(dfinal_state * final_state) for
    ``selective_forward`` with the same inputs and options (ssd_selective_backward).

    Returns a dict: dx, ddt, dB, dC and, with z, dz (dense, in x's type), dA
    [E, N] and dD [E] float32, dinit (float32 [Bt, E, N], None if not
    want_dinit) and, when dt_bias is given, ddt_bias [E] float32.
    """
    p, st, opts, G, N = _selective_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    if x.dim() != 3:
        raise ValueError("x must be [Bt, L, E]")
    _required(dy=dy)
    Bt, L, E = x.shape
    yp = _param(dy, "dy", (Bt, L, E), x, x.dtype)
    ip = _param(init_state, "init_state", (Bt, E, N), x)
    fp = _param(dfinal_state, "dfinal_state", (Bt, E, N), x)
    _on_gpu(x)
    code = dtype_code(x.dtype)
    new = lambda shape, dtype=_f32: x.new_empty(shape, dtype=dtype)  # noqa: E731
    out = {"dx": new((Bt, L, E), x.dtype), "ddt": new((Bt, L, E), x.dtype), "dA": new((E, N)),
           "dB": new((Bt, L, G, N), x.dtype), "dC": new((Bt, L, G, N), x.dtype), "dD": new((E,)),
           "dinit": new((Bt, E, N)) if want_dinit else None}
    if z is not None:
        out["dz"] = new((Bt, L, E), x.dtype)
    if dt_bias is not None:
        out["ddt_bias"] = new((E,))
    ptr = lambda k: out[k].data_ptr() if out.get(k) is not None else None  # noqa: E731
    need = _native.lib.ssd_selective_backward_workspace_size(Bt, L, E, G, N, code)
    keep, ws, ws_bytes = _workspace(workspace, need, x)
    _call(_native.lib.ssd_selective_backward, "ssd_selective_backward", x.device, *p, ip, yp, fp, Bt,
          L, E, G, N, code, ptr("dx"), ptr("ddt"), ptr("dA"), ptr("dB"), ptr("dC"), ptr("dD"),
          ptr("dz"), ptr("dinit"), ptr("ddt_bias"), ws, ws_bytes, st, opts)
    return out


def selective_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                   dt_limit=None):
    """One token of ``selective_forward`` for every sequence (ssd_selective_step):
    x, dt, z [Bt, E], B, C [Bt, G, N]; ``state`` [Bt, E, N] float32,
    selective_forward's final_state at first, is updated in place. Returns y [Bt, E].
    """
    p, st, opts, G, N = _selective_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    if x.dim() != 2:
        raise ValueError("x must be [Bt, E]")
    _required(state=state)
    Bt, E = x.shape
    sp = _param(state, "state", (Bt, E, N), x)
    _on_gpu(x)
    y = x.new_empty((Bt, E))
    _call(_native.lib.ssd_selective_step, "ssd_selective_step", x.device, sp, *p, Bt, E, G, N,
          dtype_code(x.dtype), y.data_ptr(), st, opts)
    return y


# ---- normalisation ---------------------------------------------------------------

def _rows(t, name):
    """(rows, elements between rows) of a tensor whose leading axes are one run of
    rows in memory, however far apart."""
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one axis")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    D = t.shape[-1]
    if D > 0x7fffffff:  # (rows are a long long)
        raise ValueError(f"{name}'s width must be below 2^31, got {D}")
    if t.is_contiguous():
        return (t.numel() // D if D else 0), D
    rows, step = 1, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != step * rows:
            raise ValueError(f"{name}'s rows must be evenly spaced in memory")
        rows *= size
    return rows, D if step is None else step


def norm_forward(x, weight, bias=None, residual=None, z=None, eps=1e-5, rms=False,
                 return_stats=False):
    """Layer norm (or with rms its root-mean-square form, without the mean) of
    the rows of x, of x + residual, or of x * silu(z) (ssd_norm_forward).

    x [..., D] float32 or bfloat16, D at most 16384, rows evenly spaced (a
    slice of a wider projection is fine); weight and bias [D] float32; residual
    like x, in x's type or float32; z like x (not together with residual).
    Returns y like x, dense; with residual (y, the sum in residual's type); with
    return_stats also the rows' mean (None if rms) and reciprocal standard
    deviation, float32, as norm_backward takes them. With a norm of the
    block's output, layer scale, a gate beside the residual or dropout: ``block_norm_forward``.
    """
    _required(x=x, weight=weight)
    rows, step = _rows(x, "x")
    D = x.shape[-1]
    wp = _param(weight, "weight", (D,), x)
    bp = _param(bias, "bias", (D,), x)
    rp = zp = None
    zstep, rcode = 0, 0
    if residual is not None:
        if z is not None:
            raise ValueError("residual and z exclude each other")
        if residual.dtype != _f32 and residual.dtype != x.dtype:
            raise TypeError(f"residual must be float32 or {x.dtype}, got {residual.dtype}")
        rp = _param(residual, "residual", x.shape, x, residual.dtype)
        rcode = dtype_code(residual.dtype)
    if z is not None:
        zp = _slice(z, "z", x.shape, x)
        zstep = _rows(z, "z")[1]
    _on_gpu(x)
    code = dtype_code(x.dtype)
    y = x.new_empty(x.shape)
    total = mean = rstd = None
    if residual is not None:
        total = torch.empty_like(residual)
    if return_stats:
        rstd = x.new_empty(x.shape[:-1], dtype=_f32)
        if not rms:
            mean = torch.empty_like(rstd)
    _call(_native.lib.ssd_norm_forward, "ssd_norm_forward", x.device, x.data_ptr(), step, rp, rcode,
          zp, zstep, wp, bp, rows, D, int(rms), eps, code, y.data_ptr(),
          None if total is None else total.data_ptr(), None if mean is None else mean.data_ptr(),
          None if rstd is None else rstd.data_ptr())
    out = (y,) if total is None else (y, total)
    if return_stats:
        out += (mean, rstd)
    return out if len(out) > 1 else y


def norm_backward(dy, x, weight, mean, rstd, z=None, dresidual=None, workspace=None,
                  want_dbias=None, want_dresidual=None):
    """Gradients of ``norm_forward`` (ssd_norm_backward).

    x: norm_forward's x or, where it had a residual, the sum that it returned.
    mean (None: the rms form) and rstd: its statistics. dresidual (like x): the
    gradient that reaches that sum by the skip connection.
    Returns a dict: dx (dy's type, the gradient of norm_forward's x), dweight and
    dbias ([D] float32), dz (with z) and dresidual, the gradient of
    norm_forward's residual, in x's type. want_dbias: whether dbias is formed or
    None (default: formed where there is a mean; the rms form's bias needs True).
    want_dresidual: whether dresidual is among them (default: where one is
    given; True without one where nothing comes back by the skip connection).
    """
    _required(dy=dy, x=x, weight=weight, rstd=rstd)
    rows, step = _rows(x, "x")
    D = x.shape[-1]
    if x.dtype != _f32 and x.dtype != dy.dtype:
        raise TypeError(f"x must be float32 or {dy.dtype}, got {x.dtype}")
    yp = _param(dy, "dy", x.shape, x, dy.dtype)
    wp = _param(weight, "weight", (D,), x)
    mp = _param(mean, "mean", x.shape[:-1], x)
    sp = _param(rstd, "rstd", x.shape[:-1], x)
    rp = _param(dresidual, "dresidual", x.shape, x, x.dtype)
    zp, zstep = None, 0
    want_dbias = mean is not None if want_dbias is None else bool(want_dbias)
    want_dresidual = dresidual is not None if want_dresidual is None else bool(want_dresidual)
    if z is not None:
        if dresidual is not None or want_dresidual:
            raise ValueError("dresidual and z exclude each other")
        if x.dtype != dy.dtype:
            raise TypeError(f"x must be {dy.dtype} with z, got {x.dtype}")
        zp = _slice(z, "z", x.shape, dy)
        zstep = _rows(z, "z")[1]
    _on_gpu(x)
    code = dtype_code(dy.dtype)
    out = {"dx": torch.empty_like(dy), "dweight": torch.empty_like(weight),
           "dbias": torch.empty_like(weight) if want_dbias else None}
    if z is not None:
        out["dz"] = torch.empty_like(dy)
    if want_dresidual:
        out["dresidual"] = x.new_empty(x.shape)
    ptr = lambda k: out[k].data_ptr() if out.get(k) is not None else None  # noqa: E731
    need = _native.lib.ssd_norm_backward_workspace_size(rows, D, code, int(want_dbias))
    keep, ws, ws_bytes = _workspace(workspace, need, x)
    _call(_native.lib.ssd_norm_backward, "ssd_norm_backward", x.device, yp, x.data_ptr(), step,
          dtype_code(x.dtype), zp, zstep, wp, mp, sp, rp, rows, D, code, ptr("dx"),
          ptr("dresidual"), ptr("dz"), ptr("dweight"), ptr("dbias"), ws, ws_bytes)
    return out
