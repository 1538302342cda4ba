"""Plain 64-bit CPU forms of the convolution, the selective scan and the
normalisation, token by token, with what the tests' tolerances are made of:
next to each result the sum of the absolute values of its terms (its
magnitude), through which roundings in 32 bits reach it.

One operation in 32 bits rounds by at most U32 = 2^-24 of its result, the
hardware's exponential, logarithm and reciprocal by twice that; the final
rounding to the output's type is half a step of it (`half_step`)."""
import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(name, got, want, mag, ops, slack=0.0):
    """|got - want| <= half a step of got's type at |want|, plus ops roundings
    in 32 bits of the magnitude (which the output's rounding can carry along)."""
    got64 = got.detach().double().cpu()
    assert got64.shape == want.shape, (name, got64.shape, want.shape)
    hs = half_step(got.dtype) if got.dtype != torch.float32 else U32
    tiny = torch.finfo(got.dtype).tiny
    bound = hs * want.abs() + (1 + hs) * ops * U32 * mag + tiny + slack
    err = (got64 - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (name, "worst", float((err / bound).max()),
                                 "at", torch.nonzero(bad)[0].tolist(),
                                 float(got64[bad][0]), float(want[bad][0]))


def silu(v):
    return v * torch.sigmoid(v)


def silu_grad(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def conv(x, weight, bias, act, init=None, cu=None):
    """(v before the activation, y, final state, magnitude of v), x [Bt, L, K]."""
    x, weight = x.double().cpu(), weight.double().cpu()
    K, W = weight.shape
    bias = torch.zeros(K, dtype=torch.float64) if bias is None else bias.double().cpu()
    spans = [(0, x.shape[1])] if cu is None else list(zip(cu[:-1], cu[1:]))
    v, mag = torch.zeros_like(x), torch.zeros_like(x)
    finals = []
    for a, b in spans:
        head = torch.zeros(x.shape[0], W - 1, K, dtype=torch.float64)
        if init is not None:
            head = init.double().cpu()
        xs = torch.cat([head, x[:, a:b]], 1)
        for t in range(a, b):
            win = xs[:, t - a:t - a + W].transpose(1, 2)  # [Bt, K, W]
            v[:, t] = bias + (win * weight).sum(-1)
            mag[:, t] = bias.abs() + (win * weight).abs().sum(-1)
        finals.append(xs[:, b - a:])
    return v, silu(v) if act else v, torch.cat(finals, 0), mag


def conv_grads(x, weight, bias, act, dy, init=None, dfinal=None):
    """Gradients and their magnitudes, as dicts."""
    v, _, _, _ = conv(x, weight, bias, act, init)
    x, weight, dy = x.double().cpu(), weight.double().cpu(), dy.double().cpu()
    Bt, L, K = x.shape
    W = weight.shape[1]
    head = torch.zeros(Bt, W - 1, K, dtype=torch.float64) if init is None else init.double().cpu()
    xs = torch.cat([head, x], 1)
    g = dy * (silu_grad(v) if act else 1.0)
    # the derivative's own terms: p and p v (1 - p), each at most dy (1 + |v|)
    ga = dy.abs() * (1 + v.abs())
    dxs, ma = torch.zeros_like(xs), torch.zeros_like(xs)
    dw, mw = torch.zeros_like(weight), torch.zeros_like(weight)
    for k in range(W):
        dxs[:, k:k + L] += g * weight[:, k]
        ma[:, k:k + L] += ga * weight[:, k].abs()
        dw[:, k] = (g * xs[:, k:k + L]).sum((0, 1))
        mw[:, k] = (ga * xs[:, k:k + L].abs()).sum((0, 1))
    if dfinal is not None:
        dxs[:, L:] += dfinal.double().cpu()
        ma[:, L:] += dfinal.double().cpu().abs()
    return ({"dx": dxs[:, W - 1:], "dinit": dxs[:, :W - 1], "dweight": dw, "dbias": g.sum((0, 1))},
            {"dx": ma[:, W - 1:], "dinit": ma[:, :W - 1], "dweight": mw, "dbias": ga.sum((0, 1))})


def norm(x, weight, bias, rms, eps, z=None):
    """(y, mean, rstd, magnitude of y), rows in the last axis."""
    x, weight = x.double().cpu(), weight.double().cpu()
    u = x if z is None else x * silu(z.double().cpu())
    m = torch.zeros_like(u[..., :1]) if rms else u.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + eps)
    b = torch.zeros_like(weight) if bias is None else bias.double().cpu()
    y = (u - m) * rstd * weight + b
    mag = (u.abs() + u.abs().mean(-1, keepdim=True)) * rstd * weight.abs() + b.abs()
    return y, m[..., 0], rstd[..., 0], mag


def norm_grads(dy, x, weight, rms, eps, z=None, dres=None):
    """Gradients (dx is also the stream's) and magnitudes."""
    dy, x, w = dy.double().cpu(), x.double().cpu(), weight.double().cpu()
    zd = None if z is None else z.double().cpu()
    u = x if z is None else x * silu(zd)
    m = torch.zeros_like(u[..., :1]) if rms else u.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + eps)
    n = (u - m) * r
    na = (u.abs() + (0 if rms else u.abs().mean(-1, keepdim=True))) * r
    dn = dy * w
    du = dn - n * (dn * n).mean(-1, keepdim=True)
    da = dn.abs() + na * (dn.abs() * na).mean(-1, keepdim=True)
    if not rms:
        du = du - dn.mean(-1, keepdim=True)
        da = da + dn.abs().mean(-1, keepdim=True)
    du, da = du * r, da * r
    lead = tuple(range(dy.dim() - 1))
    out = {"dweight": (dy * n).sum(lead), "dbias": dy.sum(lead)}
    mag = {"dweight": (dy.abs() * na).sum(lead), "dbias": dy.abs().sum(lead)}
    if z is not None:
        out["dz"], mag["dz"] = du * x * silu_grad(zd), da * x.abs() * (1 + zd.abs())
        du, da = du * silu(zd), da * zd.abs()
    if dres is not None:
        du, da = du + dres.double().cpu(), da + dres.double().cpu().abs()
    out["dx"], mag["dx"] = du, da
    return out, mag
