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


def selective(x, dt, A, B, C, D=None, z=None, init=None, bias=None, use_softplus=False, limit=None,
              grads=None):
    """The selective scan token by token: dict of y and final with their error
    bounds (key + "_err"), and with grads = (dy, dfinal or None) every gradient.

    The bounds follow the recurrence. A step size is off by kd = 10 + 2 |v|
    roundings of itself through softplus (1 for the bias, 2 |v| for the
    exponent, the rest for e^-|v|, log, reciprocal and sums), else 2; a decay
    exp(dt A) by (kd + 4) |dt A| + 2 of itself, an input term by kd + 3. So with
    H the recurrence of absolute values, E_t = a (E_{t-1} + ka H_{t-1}) + ku |u B|,
    and one rounding of H_t per step. Backward the same for the adjoint, whose
    products with the states take both errors."""
    d64 = lambda t: None if t is None else t.detach().double().cpu()  # noqa: E731
    x, dt, A, B, C, D, z, init, bias = map(d64, (x, dt, A, B, C, D, z, init, bias))
    Bt, L, E = x.shape
    N, G = A.shape[1], B.shape[2]
    each = E // G
    v = dt if bias is None else dt + bias
    delta, slope, kd = v, torch.ones_like(v), torch.full_like(v, 2.0)
    if use_softplus:
        delta, slope, kd = softplus(v), torch.sigmoid(v), 10 + 2 * v.abs()
    if limit is not None:
        slope = slope * ((delta >= limit[0]) & (delta <= limit[1]))
        delta = delta.clamp(*limit)
    D = torch.zeros(E, dtype=torch.float64) if D is None else D
    h = torch.zeros(Bt, E, N, dtype=torch.float64) if init is None else init.clone()
    H, Er = h.abs(), torch.zeros_like(h)
    exp = lambda m, t: m[:, t].repeat_interleave(each, 1)  # noqa: E731
    hs, Hs, Ers, ys, ym = [h], [H], [Er], torch.zeros_like(x), torch.zeros_like(x)
    for t in range(L):
        d, k = delta[:, t, :, None], kd[:, t, :, None]
        a = torch.exp(d * A)
        u = d * x[:, t, :, None] * exp(B, t)
        Er = a * (Er + ((k + 4) * (d * A).abs() + 3) * H) + (k + 4) * u.abs()
        h, H = a * h + u, a * H + u.abs()
        Er = Er + H
        ys[:, t] = (h * exp(C, t)).sum(-1) + D * x[:, t]
        ym[:, t] = ((Er + (N + 2) * H) * exp(C, t).abs()).sum(-1) + 3 * (D * x[:, t]).abs()
        hs.append(h), Hs.append(H), Ers.append(Er)
    gate = torch.ones_like(x) if z is None else silu(z)
    y = ys * gate
    kz = 0.0 if z is None else 8 + 2 * z.abs()
    out = {"y": y, "y_err": (ym + ys.abs() * kz) * gate.abs() + y.abs(), "final": h, "final_err": Er}
    if grads is None:
        return out
    dy, dfinal = map(d64, grads)
    # every product below is off by at most the sum of its factors' errors and a few roundings
    dys, dye = dy * gate, (dy * gate).abs() * (kz + 1)
    if z is not None:
        out["dz"] = dy * ys * silu_grad(z)
        out["dz_err"] = dy.abs() * (1 + z.abs()) * (ym + ys.abs() * (kz + 8))
    g = torch.zeros_like(h) if dfinal is None else dfinal.clone()
    ga, ge = g.abs(), torch.zeros_like(g)
    zero = {"dx": torch.zeros_like(x), "ddt": torch.zeros_like(x), "dB": torch.zeros_like(B),
            "dC": torch.zeros_like(C), "dA": torch.zeros_like(A)}
    out.update({k: t.clone() for k, t in zero.items()}, **{k + "_err": t.clone() for k, t in zero.items()})
    group = lambda m: m.unflatten(1, (G, each)).sum(2)  # noqa: E731
    for t in reversed(range(L)):
        d, k, xt, Bt_ = delta[:, t, :, None], kd[:, t, :, None], x[:, t, :, None], exp(B, t)
        term = dys[:, t, :, None] * exp(C, t)
        g, ge = g + term, ge + dye[:, t, :, None] * exp(C, t).abs() + ga + 2 * term.abs()
        ga = ga + term.abs()
        a = torch.exp(d * A)
        ka = (k + 4) * (d * A).abs() + 3
        out["dC"][:, t] = group(hs[t + 1] * dys[:, t, :, None])
        out["dC_err"][:, t] = group((Ers[t + 1] + (each + 4) * Hs[t + 1]) * dys[:, t, :, None].abs()
                                    + Hs[t + 1] * dye[:, t, :, None])
        out["dB"][:, t] = group(g * d * xt)
        out["dB_err"][:, t] = group((ge + (k + each + 4) * ga) * (d * xt).abs())
        gB, gBe = (g * Bt_).sum(-1), ((ge + (N + 4) * ga) * Bt_.abs()).sum(-1)
        out["dx"][:, t] = gB * d[..., 0] + D * dys[:, t]
        out["dx_err"][:, t] = (gBe + (k[..., 0] + 2) * gB.abs()) * d[..., 0].abs() + (D * dys[:, t]).abs() * 3 + D.abs() * dye[:, t]
        q, qa, qe = a * hs[t], a * Hs[t], a * (Ers[t] + (ka + 2) * Hs[t])
        # a h_{t-1} may be formed from h_t - dt x B_t, whose own error is h_t's
        qe = qe + Ers[t + 1] + 2 * Hs[t + 1] + (k + 4) * (d * xt * Bt_).abs()
        back, backe = g * q, ge * qa + ga * qe + 4 * ga * qa
        out["ddt"][:, t] = (xt[..., 0] * gB + (back * A).sum(-1)) * slope[:, t]
        out["ddt_err"][:, t] = (xt[..., 0].abs() * (gBe + 3 * gB.abs()) + ((backe + (N + 4) * ga * qa) * A.abs()).sum(-1)
                                + (k[..., 0] + 8) * (xt[..., 0].abs() * gB.abs() + (back * A).abs().sum(-1)))
        out["dA"] += (back * d).sum(0)
        out["dA_err"] += ((backe + (k + Bt * L + 4) * ga * qa) * d).sum(0)
        g, ga, ge = a * g, a * ga, a * (ge + (ka + 2) * ga)
    out["dinit"], out["dinit_err"] = g, ge + ga
    out["dD"], out["dD_err"] = (dys * x).sum((0, 1)), ((dye + (Bt * L + 2) * dys.abs()) * x.abs()).sum((0, 1))
    out["ddt_bias"] = out["ddt"].sum((0, 1))
    out["ddt_bias_err"] = (out["ddt_err"] + Bt * L * out["ddt"].abs()).sum((0, 1))
    return out
