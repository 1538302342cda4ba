"""Plain 64-bit CPU forms of the gated recurrence, the block norm and dropout, with
the errors that 32 bits may make of them (in units of layer_refs.U32, one rounding).

Roundings counted throughout: one for a product or a sum, two for the hardware's
exponential, reciprocal and square roots (1 ulp). An exponent's own rounding reaches the
exponential times the exponent, so sigmoid(v) is off by at most 8 + 2 |v|, softplus(v) by
10 + 2 |v| of itself."""
import numpy as np
import torch

import layer_refs as R

JOINS = 60  # sums and products that join strands (4), wavefronts (4) and a group's tiles (16), each way
KEEP = 16   # tokens between the states that the forward keeps


def _d(t):
    return None if t is None else t.detach().double().cpu()


def recurrence(x, r, i=None, decay=None, z=None, init=None, c=8.0, cu=None, grads=None):
    """Token by token: dict of y, final and states with their errors (key + "_err"), and with
    grads = (dy, dfinal or None) every gradient.

    log a is off by kl = 13 + 2 |decay| (its rate) + 8 + 2 |r| (the gate) + 1 of itself, a
    by ka = kl |log a| + 3. 1 - a^2 is off by kl + 17 at most: relative to itself it moves
    at most as log a does, the series has 8 roundings, and 1 - a^2 without it (a^2 below 0.78) 4 *
    0.78 / 0.22 + 1; its root by half of that and 2. Per token the state takes ka + 2 of
    the decayed one (maps of several tokens multiply their a), the input term's error and one
    rounding; the joins of the maps on top."""
    x, r, i, decay, z, init = map(_d, (x, r, i, decay, z, init))
    Bt, L, E = x.shape
    gated = decay is not None
    spans = [(0, L)] if cu is None else list(zip(cu[:-1], cu[1:]))
    first = {a for a, b in spans if b > a} if cu is not None else set()
    dy, dfinal = map(_d, grads or (None, None))
    if cu is not None:  # padding: no sequence's, as if it held zeros and began anew with every token
        pad = [t for t in range(L) if t < cu[0] or t >= cu[-1]]
        first |= set(pad)
        x, r, i, z, dy = (t if t is None else t.index_fill(1, torch.tensor(pad, dtype=torch.int64), 0.0)
                          for t in (x, r, i, z, dy))
    last = {b - 1: k for k, (a, b) in enumerate(spans) if b > a}
    if gated:
        sr, si = torch.sigmoid(r), torch.sigmoid(i)
        rate = -c * R.softplus(decay)
        la = rate * sr
        kr, ki = 8 + 2 * r.abs(), 8 + 2 * i.abs()
        kl = 14 + 2 * decay.abs() + kr
        a = torch.exp(la)
        b = torch.sqrt(-torch.expm1(2 * la))
        kb = (kl + 17) / 2 + 2
        u, ku = b * si * x, kb + ki + 3
    else:
        la, a, u = r, torch.exp(r), x
        kl, ku = torch.full_like(r, 2.0), torch.zeros_like(r)
    # (an exponent of -inf gives 0 exactly)
    ka = torch.where(torch.isinf(la), 0.0, kl * la.abs()) + 3
    zero = torch.zeros(Bt, E, dtype=torch.float64)
    h = zero if init is None else init
    H, Er = h.abs(), zero
    # states, their magnitudes and errors before and behind every token
    before, after = torch.zeros(2, 3, Bt, L, E, dtype=torch.float64)
    states, states_err = torch.zeros(2, Bt, -(-L // KEEP), E, dtype=torch.float64)
    final, final_err = torch.zeros(2, len(spans), E, dtype=torch.float64)
    for t in range(L):
        if t % KEEP == 0:
            states[:, t // KEEP], states_err[:, t // KEEP] = h, Er + JOINS * H
        if t in first:
            h, H, Er = zero, zero, zero
        before[0][:, t], before[1][:, t], before[2][:, t] = h, H, Er
        Er = a[:, t] * (Er + (ka[:, t] + 2) * H) + (ku[:, t] + 1) * u[:, t].abs()
        h, H = a[:, t] * h + u[:, t], a[:, t] * H + u[:, t].abs()
        Er = Er + H
        after[0][:, t], after[1][:, t], after[2][:, t] = h, H, Er
        if cu is not None and t in last:
            final[last[t]], final_err[last[t]] = h[0], (Er + JOINS * H)[0]
    if cu is None:
        final, final_err = h, Er + JOINS * H
    gate, kz = torch.ones_like(x), torch.zeros_like(x)
    if z is not None:
        gate, kz = R.silu(z), 9 + 2 * z.abs()
    hy, Hy, Ey = after
    Ey = Ey + JOINS * Hy
    out = {"y": hy * gate, "y_err": (Ey + kz * Hy) * gate.abs(), "final": final, "final_err": final_err,
           "states": states, "states_err": states_err}
    if grads is None:
        return out
    if z is not None:
        out["dz"] = dy * hy * R.silu_grad(z)
        out["dz_err"] = dy.abs() * (1 + z.abs()) * (Ey + (kz + 8) * Hy)
    gy, gye = dy * gate, (dy * gate).abs() * (kz + 1)
    g = zero if dfinal is None or cu is not None else dfinal
    G, Eg = g.abs(), zero
    for k in ("dx", "dr", "di") if gated else ("dx", "dr"):
        out[k], out[k + "_err"] = torch.zeros_like(x), torch.zeros_like(x)
    W, We, Wa = zero.clone(), zero.clone(), zero.clone()
    for t in reversed(range(L)):
        if cu is not None and dfinal is not None and t in last:
            g, G = g + dfinal[last[t]], G + dfinal[last[t]].abs()
        g, Eg, G = g + gy[:, t], Eg + gye[:, t], G + gy[:, t].abs()
        Eg = Eg + 2 * G
        e = Eg + JOINS * G
        at, kat, hp, Hp, Ep = a[:, t], ka[:, t], *(v[:, t] for v in before)
        Ep = Ep + JOINS * Hp
        back, backe, backa = g * at * hp, at * (G * Ep + e * Hp + (kat + 4) * G * Hp), at * G * Hp
        if gated:
            bt, st, xt, lt = b[:, t], si[:, t], x[:, t], la[:, t]
            dx, dxa = g * bt * st, G * bt * st
            dxe = e * bt * st + dxa * (kb[:, t] + ki[:, t] + 3)
            out["dx"][:, t], out["dx_err"][:, t] = dx, dxe
            out["di"][:, t] = dx * xt * (1 - st)
            out["di_err"][:, t] = dxe * xt.abs() * (1 - st) + dxa * xt.abs() * (ki[:, t] * st + 4)
            q = torch.where(bt > 0, lt / bt, 0) * st * xt * at * at
            w = back * lt - g * q
            wa = backa * lt.abs() + G * q.abs()
            we = (backe + backa * (kl[:, t] + 3)) * lt.abs() + q.abs() * (
                e + G * (ki[:, t] + 2 * kat + kl[:, t] + kb[:, t] + 8)) + 2 * wa
            out["dr"][:, t] = w * (1 - sr[:, t])
            out["dr_err"][:, t] = we * (1 - sr[:, t]) + wa * (kr[:, t] * sr[:, t] + 3)
            W, We, Wa = W + w, We + we, Wa + wa
        else:
            out["dx"][:, t], out["dx_err"][:, t] = g, e
            out["dr"][:, t], out["dr_err"][:, t] = back, backe
        if t in first:
            g, G, Eg = zero, zero, zero
        else:
            g, G, Eg = at * g, at * G, at * (Eg + (kat + 2) * G) + at * G
    out["dinit"], out["dinit_err"] = g, Eg + (JOINS + 2) * G
    if gated:
        k = torch.where(decay < -30, 1.0, torch.sigmoid(decay) / R.softplus(decay).clamp(min=1e-300))
        out["ddecay"] = k * W.sum(0)
        # 22 + 4 |decay|: sigmoid, softplus, their quotient and the product
        out["ddecay_err"] = k * (We.sum(0) + (Bt * L + JOINS + 22 + 4 * decay.abs()) * Wa.sum(0))
    return out


# ---- dropout --------------------------------------------------------------------------

def philox(counter, key):
    """Philox 4x32-10 of counters [..., 4] and a key of two words, in 64-bit integers."""
    x = [np.asarray(counter)[..., k].astype(np.uint64) for k in range(4)]
    k0, k1 = key
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(q >> half) ^ x[1] ^ np.uint64(k0), q & low, (p >> half) ^ x[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    return np.stack(x, -1)


def kept(rows, width, p, seed, offset, first=0):
    """Which elements of [rows, width] stay, from row `first` on."""
    groups = -(-width // 8)
    counter = np.zeros((rows, groups, 4), np.uint64)
    counter[..., 0] = np.arange(groups)
    counter[..., 1] = first + np.arange(rows)[:, None]
    counter[..., 2], counter[..., 3] = offset % 2 ** 32, offset >> 32
    w = philox(counter, (seed % 2 ** 32, seed >> 32))
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(rows, -1)[:, :width]
    return torch.from_numpy(bits.astype(np.int64) >= int(np.floor(p * 65536 + 0.5)))


def share(p):
    """What a kept element is multiplied with."""
    t = np.floor(p * 65536 + 0.5)
    return 65536 / (65536 - t) if t < 65536 else 0.0


def dropped(x, p, rng):
    k = kept(x.numel() // x.shape[-1], x.shape[-1], p, *rng).view(x.shape)
    return torch.where(k, _d(x) * share(p), 0.0)


# ---- block norm -------------------------------------------------------------------------

def _norm(u, rms, eps):
    """n, rstd and the magnitude of n."""
    m = torch.zeros_like(u[..., :1]) if rms else u.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + eps)
    return (u - m) * r, r, (u.abs() + (0 if rms else u.abs().mean(-1, keepdim=True))) * r


def _norm_grad(dn, da, n, na, r, rms):
    """The gradient of u and its magnitude, from the gradient of n and its."""
    du = dn - n * (dn * n).mean(-1, keepdim=True)
    ua = da + na * (da * na).mean(-1, keepdim=True)
    if not rms:
        du, ua = du - dn.mean(-1, keepdim=True), ua + da.mean(-1, keepdim=True)
    return du * r, ua * r


class Block:
    """The block norm of x and residual (rows in the last axis), all in 64 bits. After the
    construction: total and its magnitude total_mag; y(total) and grads(...)."""

    def __init__(self, x, residual, weight=None, bias=None, post_weight=None, post_bias=None, scale=None, z=None,
                 alpha=1.0, beta=1.0, p=0.0, rng=None, eps=1e-5, rms=False):
        self.x, res, self.w, self.b, self.pw, self.pb, self.scale, self.z = map(
            _d, (x, residual, weight, bias, post_weight, post_bias, scale, z))
        self.alpha, self.beta, self.eps, self.rms = alpha, beta, eps, rms
        one = torch.ones_like(self.x)
        v, va = self.x, self.x.abs()
        if self.pw is not None:
            self.n, self.r, self.na = _norm(self.x, rms, eps)
            v, va = self.n * self.pw, self.na * self.pw.abs()
            if self.pb is not None:
                v, va = v + self.pb, va + self.pb.abs()
        self.v, self.va = v, va
        self.k = one if self.scale is None else one * self.scale
        self.gate = one if self.z is None else R.silu(self.z)
        self.drop = one
        if p:
            self.drop = kept(one.numel() // one.shape[-1], one.shape[-1], p, *rng).view(one.shape).double() * share(p)
        m = self.k * self.gate * self.drop
        self.total = alpha * res + beta * v * m
        self.total_mag = abs(alpha) * res.abs() + abs(beta) * va * m.abs()

    def y(self, total):
        """The norm before the next block, of the stream as it was kept, and its magnitude."""
        n, _, na = _norm(_d(total), self.rms, self.eps)
        y, ya = n * self.w, na * self.w.abs()
        return (y, ya) if self.b is None else (y + self.b, ya + self.b.abs())

    def grads(self, dy, dsum, total):
        """Gradients and their magnitudes, as dicts."""
        dy, dsum = _d(dy), _d(dsum)
        lead = tuple(range(self.x.dim() - 1))
        out, mag = {}, {}
        ds, da = (torch.zeros_like(self.x),) * 2 if dsum is None else (dsum, dsum.abs())
        if self.w is not None:
            n, r, na = _norm(_d(total), self.rms, self.eps)
            g, ga = _norm_grad(dy * self.w, (dy * self.w).abs(), n, na, r, self.rms)
            ds, da = ds + g, da + ga
            out["dweight"], mag["dweight"] = (dy * n).sum(lead), (dy.abs() * na).sum(lead)
            if self.b is not None:
                out["dbias"], mag["dbias"] = dy.sum(lead), dy.abs().sum(lead)
        out["dresidual"], mag["dresidual"] = self.alpha * ds, abs(self.alpha) * da
        db, ba = self.beta * self.drop * ds, abs(self.beta) * self.drop * da
        if self.z is not None:
            out["dz"] = db * self.v * self.k * R.silu_grad(self.z)
            mag["dz"] = ba * self.va * self.k.abs() * (1 + self.z.abs())
        e, ea = db * self.gate, ba * self.gate.abs()
        if self.scale is not None:
            out["dscale"], mag["dscale"] = (e * self.v).sum(lead), (ea * self.va).sum(lead)
        dv, dva = e * self.k, ea * self.k.abs()
        if self.pw is not None:
            out["dpost_weight"], mag["dpost_weight"] = (dv * self.n).sum(lead), (dva * self.na).sum(lead)
            if self.pb is not None:
                out["dpost_bias"], mag["dpost_bias"] = dv.sum(lead), dva.sum(lead)
            dv, dva = _norm_grad(dv * self.pw, dva * self.pw.abs(), self.n, self.na, self.r, self.rms)
        out["dx"], mag["dx"] = dv, dva
        return out, mag
