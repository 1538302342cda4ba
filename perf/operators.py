"""The operators around the state-space layers, as cases to be measured: the
short causal convolution, the selective scan with one decay rate per channel
and state, and the normalisation, for prompts, single tokens and training.

``run`` computes a case with elementary torch operations, or (``own``) with the
library's entry points. ``exact`` computes the same from the definition in 64
bits, token by token.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
# tokens per chunk and chunks per group of the plain scan (see _linear_scan)
Q, GROUP = 8, 16


def listed():
    return [
        # prompts of a Mamba-2 2.7B layer: x, B and C are convolved together, a slice of the
        # input projection (next to the gate and the step sizes), and leave as three tensors
        dict(name="conv prompt", op="conv", mode="forward", batch=8, seqlen=2048, split="5120,64,64",
             width=4, dtype="bf16", init=0, pad=5200),
        # short documents packed into one token axis, as prefill batches and pre-training make them
        dict(name="conv packed", op="conv", mode="packed", batch=1, seqlen=16384, split="5120,64,64",
             width=4, dtype="bf16", init=0, pad=0),
        # a continued sequence of odd length in float32, with gradients
        dict(name="conv train f32", op="conv", mode="train", batch=3, seqlen=1021, split="1312",
             width=3, dtype="f32", init=1, pad=0),
        # one token for each of 256 sequences in decoding (8 groups of B and C, state 128)
        dict(name="conv step", op="conv", mode="step", batch=256, seqlen=1, split="5120,1024,1024",
             width=4, dtype="bf16", init=1, pad=0),
        # one long prompt: few channels to fill the GPU with, so the token axis has to be split
        dict(name="scan prompt", op="scan", mode="forward", batch=1, seqlen=8192, channels=5120,
             state=16, groups=1, dtype="bf16", init=0, gate=1, pad=160),
        # a training step of a layer of the same width
        dict(name="scan train", op="scan", mode="train", batch=4, seqlen=2048, channels=5120, state=16,
             groups=1, dtype="bf16", init=0, gate=1, pad=160),
        # odd sizes in float32: a state that is no power of two, two groups, a given initial state
        dict(name="scan train f32", op="scan", mode="train", batch=2, seqlen=777, channels=1000, state=24,
             groups=2, dtype="f32", init=1, gate=0, pad=0),
        # one token for each of 256 sequences, and for a single one
        dict(name="scan step", op="scan", mode="step", batch=256, seqlen=1, channels=5120, state=16,
             groups=1, dtype="bf16", init=1, gate=1, pad=160),
        dict(name="scan step one", op="scan", mode="step", batch=1, seqlen=1, channels=5120, state=16,
             groups=1, dtype="bf16", init=1, gate=1, pad=160),
        # the normalisation before every block, over the sum of branch and float32 residual stream
        dict(name="norm train", op="norm", mode="train", rows=16384, width=2560, dtype="bf16", rms=0,
             residual="f32", gate=0),
        # the gated root-mean-square form behind the scan, an odd number of rows
        dict(name="norm train gated", op="norm", mode="train", rows=4099, width=5120, dtype="bf16", rms=1,
             residual="", gate=1),
        # one token of a few sequences
        dict(name="norm step", op="norm", mode="forward", rows=4, width=2560, dtype="bf16", rms=1,
             residual="bf16", gate=0),
    ]


def _loguniform(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _init(rng, mode):
    return {"step": 1, "packed": 0}.get(mode, rng.randint(0, 1))


def draw(rng):
    op = rng.choice(["conv", "scan", "norm"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "norm":
        width = _loguniform(rng, 16, 16384)
        gate = rng.randint(0, 1)
        return dict(op=op, mode=rng.choice(["forward", "train"]), rows=_loguniform(rng, 1, min(16384, (1 << 25) // width)),
                    width=width, dtype=dtype, rms=rng.randint(0, 1), gate=gate,
                    residual="" if gate else rng.choice(["", "f32", dtype]))
    mode = rng.choice(["forward", "train", "step"] + (["packed"] if op == "conv" else []))
    batch = _loguniform(rng, 1, 256 if mode == "step" else 1 if mode == "packed" else 8)
    if op == "conv":
        channels = _loguniform(rng, 16, 8192)
        parts = [channels]
        if rng.randint(0, 1) and channels >= 64:
            side = rng.randint(1, channels // 8)
            parts = [channels - 2 * side, side, side]
        seqlen = 1 if mode == "step" else _loguniform(rng, 1, min(16384, (1 << 25) // (batch * channels)))
        return dict(op=op, mode=mode, batch=batch, seqlen=seqlen, split=",".join(map(str, parts)),
                    width=rng.randint(2, 4), dtype=dtype, init=_init(rng, mode),
                    pad=rng.choice([0, 0, 64, 3]))
    state, groups = _loguniform(rng, 1, 64), rng.choice([1, 1, 2, 4])
    channels = groups * _loguniform(rng, 16, 8192 // groups)
    most = (1 << 28) // (batch * channels * state)
    seqlen = 1 if mode == "step" else _loguniform(rng, 1, max(1, min(8192, most)))
    return dict(op=op, mode=mode, batch=batch, seqlen=seqlen, channels=channels, state=state, groups=groups,
                dtype=dtype, init=_init(rng, mode), gate=rng.randint(0, 1), pad=rng.choice([0, 0, 96, 5]))


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)

    def uniform(*shape, lo, hi):
        return torch.rand(*shape, generator=g, device=DEV).mul_(hi - lo).add_(lo)

    t = _type(case["dtype"])
    s = dict(case=dict(case))
    if case["op"] == "conv":
        parts = [int(v) for v in case["split"].split(",")]
        K, W, Bt, L = sum(parts), case["width"], case["batch"], case["seqlen"]
        s["parts"] = parts
        lead = (Bt,) if case["mode"] == "step" else (Bt, L)
        s["x"] = normal(*lead, K + case["pad"], dtype=t)[..., case["pad"]:]
        s["weight"] = uniform(K, W, lo=-W ** -0.5, hi=W ** -0.5)
        s["bias"] = uniform(K, lo=-W ** -0.5, hi=W ** -0.5)
        s["init"] = normal(Bt, W - 1, K, dtype=t) if case["init"] else None
        if case["mode"] == "packed":
            r = torch.Generator().manual_seed(int(seed))
            lengths = torch.exp(torch.rand(1 + L // 300, generator=r, dtype=torch.float64) * math.log(2049))
            cu = torch.cat([torch.zeros(1), (lengths.cumsum(0) / lengths.sum() * L).round()])
            s["cu"] = cu.to(torch.int32).to(DEV)
        if case["mode"] == "train":
            s["dy"] = [normal(Bt, L, k, dtype=t) for k in parts]
    elif case["op"] == "scan":
        Bt, L, E, N, G, pad = (case[k] for k in ("batch", "seqlen", "channels", "state", "groups", "pad"))
        lead = (Bt,) if case["mode"] == "step" else (Bt, L)
        s["x"] = normal(*lead, E, dtype=t)
        s["dt"] = normal(*lead, E, dtype=t, scale=0.5)
        s["dt_bias"] = uniform(E, lo=-6.5, hi=-3.0)
        s["A"] = -torch.exp(uniform(E, N, lo=0.0, hi=math.log(16.0)))
        # B and C come out of one projection, behind the step sizes' low-rank part
        bc = normal(*lead, pad + 2 * G * N, dtype=t, scale=N ** -0.5)
        s["B"] = bc[..., pad:pad + G * N].unflatten(-1, (G, N))
        s["C"] = bc[..., pad + G * N:].unflatten(-1, (G, N))
        s["D"] = normal(E)
        # the gate is the second half of the input projection
        s["z"] = normal(*lead, 2 * E, dtype=t)[..., E:] if case["gate"] else None
        s["init"] = normal(Bt, E, N, scale=0.1) if case["init"] else None
        if case["mode"] == "train":
            s["dy"] = normal(Bt, L, E, dtype=t)
    else:
        R, D = case["rows"], case["width"]
        s["x"] = normal(R, D, dtype=t)
        s["weight"] = 1.0 + normal(D, scale=0.1)
        s["bias"] = None if case["rms"] else normal(D, scale=0.1)
        s["residual"] = normal(R, D, dtype=_type(case["residual"])) if case["residual"] else None
        s["z"] = normal(R, 2 * D, dtype=t)[:, :D] if case["gate"] else None
        if case["mode"] == "train":
            s["dy"] = normal(R, D, dtype=t)
            s["dresidual"] = normal(R, D, dtype=_type(case["residual"])) if case["residual"] else None
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[op](state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[op](state)


# ---- the library's entry points ------------------------------------------------

def _own_conv(s):
    import structured_state_space_ssd_amd as ssd
    mode, split = s["case"]["mode"], s["parts"] if len(s["parts"]) > 1 else None
    if mode == "step":
        y = ssd.conv_step(s["init"], s["x"], s["weight"], s["bias"], split=split)
        return {"y": y, "state": s["init"]}
    y, final = ssd.conv_forward(s["x"], s["weight"], s["bias"], init_state=s["init"], return_final_state=True,
                                cu_seqlens=s.get("cu"), split=split)
    out = {"y": y, "final": final}
    if mode == "train":
        g = ssd.conv_backward(s["x"], s["weight"], s["bias"], s["dy"] if split else s["dy"][0],
                              init_state=s["init"])
        out.update(dx=g["dx"], dweight=g["dweight"], dbias=g["dbias"])
        if s["init"] is not None:
            out["dinit"] = g["dinit"]
    return out


def _own_scan(s):
    import structured_state_space_ssd_amd as ssd
    mode = s["case"]["mode"]
    if mode == "step":
        y = ssd.selective_step(s["init"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], z=s["z"],
                               dt_bias=s["dt_bias"], dt_softplus=True)
        return {"y": y, "state": s["init"]}
    y, final = ssd.selective_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], z=s["z"],
                                     init_state=s["init"], return_final_state=True, dt_bias=s["dt_bias"],
                                     dt_softplus=True)
    out = {"y": y, "final": final}
    if mode == "train":
        g = ssd.selective_backward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dy"], z=s["z"],
                                   init_state=s["init"], dt_bias=s["dt_bias"], dt_softplus=True,
                                   want_dinit=s["init"] is not None)
        out.update({k: g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias")})
        if s["z"] is not None:
            out["dz"] = g["dz"]
        if s["init"] is not None:
            out["dinit"] = g["dinit"]
    return out


def _own_norm(s):
    import structured_state_space_ssd_amd as ssd
    c = s["case"]
    train = c["mode"] == "train"
    r = ssd.norm_forward(s["x"], s["weight"], s["bias"], residual=s["residual"], z=s["z"], eps=EPS,
                         rms=bool(c["rms"]), return_stats=train)
    r = r if isinstance(r, tuple) else (r,)
    out = {"y": r[0]}
    if s["residual"] is not None:
        out["sum"] = r[1]
    if train:
        g = ssd.norm_backward(s["dy"], out.get("sum", s["x"]), s["weight"], r[-2], r[-1], z=s["z"],
                              dresidual=s["dresidual"])
        out.update(dx=g["dx"], dweight=g["dweight"])
        if not c["rms"]:
            out["dbias"] = g["dbias"]
        if s["z"] is not None:
            out["dz"] = g["dz"]
        if s["residual"] is not None:
            out["dresidual"] = g["dresidual"]
    return out


# ---- plain forms: 32 bits, rounded once at the end --------------------------------

def _silu_grad(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def _plain_conv(s):
    c, parts, x = s["case"], s["parts"], s["x"]
    W, L, mode = c["width"], c["seqlen"], c["mode"]
    w = s["weight"].t()
    xs = (x[:, None] if mode == "step" else x).float()
    before = (s["init"].float() if s["init"] is not None else xs.new_zeros(xs.shape[0], W - 1, xs.shape[2]))
    xp = torch.cat([before, xs], 1)
    if mode == "packed":
        at = torch.arange(L, device=x.device)
        cu = s["cu"].long()
        since = at - cu[torch.searchsorted(cu, at, right=True) - 1]  # tokens of the sequence before this one
        pre = s["bias"] + sum(w[k] * xp[:, k:k + L] * (since >= W - 1 - k)[:, None] for k in range(W))
        rows = cu[1:, None] - (W - 1) + torch.arange(W - 1, device=x.device)
        final = torch.where((rows >= cu[:-1, None])[..., None], x[0][rows.clamp(min=0)], 0)
    else:
        pre = s["bias"] + sum(w[k] * xp[:, k:k + L] for k in range(W))
        final = xp[:, L:].to(x.dtype)
    y = (pre * torch.sigmoid(pre)).to(x.dtype)
    if mode == "step":
        y = y[:, 0]
        s["init"].copy_(final)
    y = [v.contiguous() for v in y.split(parts, -1)]
    out = {"y": tuple(y) if len(parts) > 1 else y[0]}
    if mode == "step":
        return {**out, "state": s["init"]}
    out["final"] = final
    if mode == "train":
        dpre = torch.cat([v.float() for v in s["dy"]], -1) * _silu_grad(pre)
        after = torch.nn.functional.pad(dpre, (0, 0, W - 1, W - 1))
        dxp = sum(w[k] * after[:, W - 1 - k:W - 1 - k + L + W - 1] for k in range(W))
        out["dx"] = dxp[:, W - 1:].to(x.dtype)
        out["dweight"] = torch.stack([(dpre * xp[:, k:k + L]).sum((0, 1)) for k in range(W)], 1)
        out["dbias"] = dpre.sum((0, 1))
        if s["init"] is not None:
            out["dinit"] = dxp[:, :W - 1].to(x.dtype)
    return out


def _carry(S, U, h0):
    """States entering each of n chunks (dim 1) and leaving the last one, from every chunk's
    log-decay S and its state U from zero; h0 (or None) enters the first."""
    n = S.shape[1]
    if n > GROUP:
        m = -(-n // GROUP)
        fill = (0, 0) * (S.dim() - 2) + (0, m * GROUP - n)
        S = torch.nn.functional.pad(S, fill).unflatten(1, (m, GROUP))
        U = torch.nn.functional.pad(U, fill).unflatten(1, (m, GROUP))
        inner, last = _carry(S.flatten(0, 1), U.flatten(0, 1), None)
        inner, last = inner.view(S.shape), last.view(S.shape[:2] + S.shape[3:])
        enter, end = _carry(S.sum(2), last, h0)
        P = S.cumsum(2) - S  # decay from the group's start to each chunk's
        return (inner + torch.exp(P) * enter[:, :, None]).flatten(1, 2)[:, :n], end
    P = torch.nn.functional.pad(S, (0, 0) * (S.dim() - 2) + (1, 0)).cumsum(1)
    i = torch.arange(n + 1, device=S.device)
    keep = (i[:, None] > i[None, :n]).view((n + 1, n) + (1,) * (S.dim() - 2))
    M = torch.exp((P[:, :, None] - P[:, None, 1:]).masked_fill(~keep, -torch.inf))
    H = (M * U[:, None]).sum(2)
    if h0 is not None:
        H = H + torch.exp(P) * h0[:, None]
    return H[:, :n], H[:, n]


def _linear_scan(la, v, h0):
    """h_t = exp(la_t) h_{t-1} + v_t along dim 1: every h_t, and the last. Within chunks of Q
    tokens through sums of v_t / exp(running sum of la), whose range Q keeps small; between
    chunks by _carry."""
    L = la.shape[1]
    n = -(-L // Q)
    fill = (0, 0) * (la.dim() - 2) + (0, n * Q - L)
    P = torch.nn.functional.pad(la, fill).unflatten(1, (n, Q)).cumsum(2)
    v = torch.nn.functional.pad(v, fill).unflatten(1, (n, Q))
    up = torch.exp(P)
    local = up * (v / up).cumsum(2)
    enter, end = _carry(P[:, :, -1], local[:, :, -1], h0)
    return (local + up * enter[:, :, None]).flatten(1, 2)[:, :L], end


def _plain_scan(s):
    c = s["case"]
    mode, x, A, D = c["mode"], s["x"], s["A"], s["D"]
    each = c["channels"] // c["groups"]
    v = s["dt"].float() + s["dt_bias"]
    delta = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    xf = x.float()
    # [..., E, N], one group's B and C for each of its channels
    Bf, Cf = (m.float().repeat_interleave(each, -2) for m in (s["B"], s["C"]))
    gate = 1.0
    if s["z"] is not None:
        zf = s["z"].float()
        gate = zf * torch.sigmoid(zf)
    if mode == "step":
        h = s["init"]
        h.mul_(torch.exp(delta[..., None] * A)).add_((delta * xf)[..., None] * Bf)
        y = ((h * Cf).sum(-1) + D * xf) * gate
        return {"y": y.to(x.dtype), "state": h}
    la = delta[..., None] * A
    h, final = _linear_scan(la, (delta * xf)[..., None] * Bf, s["init"])
    ys = (h * Cf).sum(-1) + D * xf
    out = {"y": (ys * gate).to(x.dtype), "final": final}
    if mode != "train":
        return out
    dy = s["dy"].float()
    if s["z"] is not None:
        out["dz"] = (dy * ys * _silu_grad(zf)).to(x.dtype)
        dy = dy * gate
    # the adjoint runs backward: g_t = dy_t C_t + exp(la_{t+1}) g_{t+1}
    later = torch.cat([la[:, 1:], torch.zeros_like(la[:, :1])], 1)
    g = _linear_scan(later.flip(1), (dy[..., None] * Cf).flip(1), None)[0].flip(1)
    first = s["init"][:, None] if s["init"] is not None else torch.zeros_like(h[:, :1])
    decayed = torch.exp(la) * torch.cat([first, h[:, :-1]], 1)
    gB = (g * Bf).sum(-1)
    gq = g * decayed
    ddelta = xf * gB + (gq * A).sum(-1)
    ddt = ddelta * torch.sigmoid(v)
    out["dx"] = (delta * gB + D * dy).to(x.dtype)
    out["ddt"] = ddt.to(x.dtype)
    out["ddt_bias"] = ddt.sum((0, 1))
    out["dA"] = (gq * delta[..., None]).sum((0, 1))
    out["dD"] = (dy * xf).sum((0, 1))
    by_group = lambda m: m.unflatten(-2, (c["groups"], each)).sum(-2).to(x.dtype)  # noqa: E731
    out["dB"] = by_group(g * (delta * xf)[..., None])
    out["dC"] = by_group(h * dy[..., None])
    if s["init"] is not None:
        out["dinit"] = torch.exp(la[:, 0]) * g[:, 0]
    return out


def _plain_norm(s):
    c, x, w = s["case"], s["x"], s["weight"]
    out = {}
    u = x.float()
    if s["residual"] is not None:
        # the stream is what is kept, so the norm reads it as it is kept
        out["sum"] = (u + s["residual"].float()).to(s["residual"].dtype)
        u = out["sum"].float()
    if s["z"] is not None:
        zf, xf = s["z"].float(), u
        gate = zf * torch.sigmoid(zf)
        u = xf * gate
    d = u if c["rms"] else u - u.mean(-1, keepdim=True)
    rstd = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    n = d * rstd
    y = n * w if s["bias"] is None else n * w + s["bias"]
    out["y"] = y.to(x.dtype)
    if c["mode"] != "train":
        return out
    dy = s["dy"].float()
    dn = dy * w
    du = dn - n * (dn * n).mean(-1, keepdim=True)
    if not c["rms"]:
        du = du - dn.mean(-1, keepdim=True)
        out["dbias"] = dy.sum(0)
    du = du * rstd
    out["dweight"] = (dy * n).sum(0)
    if s["z"] is not None:
        out["dz"] = (du * xf * _silu_grad(zf)).to(x.dtype)
        du = du * gate
    if s["residual"] is not None:
        du = du + s["dresidual"].float()
        out["dresidual"] = du.to(s["residual"].dtype)
    out["dx"] = du.to(x.dtype)
    return out


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["mode"] == "train"
    if case["op"] == "norm":
        n, D = case["rows"] * case["width"], case["width"]
        r = {"": 0, "f32": 4, "bf16": 2}[case["residual"]]
        each = 2 * e + 2 * r + e * case["gate"]  # x, y; the stream in and out; the gate
        if train:
            each += 2 * e + 2 * r + e * case["gate"]  # dy, dx; the stream's gradient in and out; dz
        return {"bytes": n * each + 4 * D * (4 if train else 2), "flops": n * (24 if train else 9)}
    if case["op"] == "conv":
        K, W = sum(int(v) for v in case["split"].split(",")), case["width"]
        n = case["batch"] * case["seqlen"] * K
        states = case["batch"] * (W - 1) * K * e
        each, flops = 2 * e, 2 * W + 5
        if train:
            each, flops = each + 2 * e, flops + 4 * W + 12
        return {"bytes": n * each + 4 * K * (W + 1) * (2 if train else 1) + states * (1 + case["init"]),
                "flops": n * flops}
    Bt, L, E, N, G = (case[k] for k in ("batch", "seqlen", "channels", "state", "groups"))
    n, bc, states = Bt * L * E, Bt * L * G * N, Bt * E * N * 4
    tensors = 3 + case["gate"]  # x, dt, y, the gate
    b, flops = n * e * tensors + 2 * bc * e + 4 * E * (N + 2) + states * (1 + case["init"]), n * (7 * N + 10)
    if train:  # dy, dx, ddt, dz, dB, dC; the parameters' gradients; the initial state's
        b += n * e * tensors + 2 * bc * e + 4 * E * (N + 2) + states * case["init"]
        flops += n * (20 * N + 20)
    return {"bytes": b, "flops": flops}


# ---- the definition in 64 bits, token by token ----------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s)


def _exact_conv(s):
    c, parts, x, w = s["case"], s["parts"], s["x"], s["weight"]
    W, mode = c["width"], c["mode"]
    if mode == "packed":
        cu = s["cu"].tolist()
        spans = [x[:, a:b] for a, b in zip(cu[:-1], cu[1:])]
    else:
        spans = [x[:, None] if mode == "step" else x]
    ys, finals = [], []
    for v in spans:
        K, L = v.shape[2], v.shape[1]
        before = s["init"] if s["init"] is not None else v.new_zeros(v.shape[0], W - 1, K)
        v = torch.cat([before, v], 1)
        finals.append(v[:, L:])
        if L == 0:  # an empty sequence
            continue
        windows = v.unfold(1, W, 1)  # [Bt, L, K, W]
        if mode == "train":
            windows = windows.clone().requires_grad_(True)
            w = w.clone().requires_grad_(True)
            bias = s["bias"].clone().requires_grad_(True)
        else:
            bias = s["bias"]
        y = torch.nn.functional.silu((windows * w).sum(-1) + bias)
        ys.append(y)
    y, final = torch.cat(ys, 1), torch.cat(finals, 0)
    out = {"final": final}
    if mode == "train":
        dwin, dw, db = torch.autograd.grad(y, (windows, w, bias), torch.cat([v.double() for v in s["dy"]], -1))
        dv = torch.zeros(y.shape[0], y.shape[1] + W - 1, y.shape[2], dtype=torch.float64, device=y.device)
        for k in range(W):
            dv[:, k:k + y.shape[1]] += dwin[..., k]
        out.update(dx=dv[:, W - 1:], dweight=dw, dbias=db)
        if s["init"] is not None:
            out["dinit"] = dv[:, :W - 1]
        y = y.detach()
    if mode == "step":
        y, out = y[:, 0], {"state": final}
    out["y"] = tuple(y.split(parts, -1)) if len(parts) > 1 else y
    return out


def _exact_scan(s):
    c = s["case"]
    mode, A, D, G = c["mode"], s["A"], s["D"], c["groups"]
    x, dt, B, C, z = (s[k][:, None] if mode == "step" and s[k] is not None else s[k] for k in ("x", "dt", "B", "C", "z"))
    Bt, L, E = x.shape
    N, each = A.shape[1], E // G
    pre = dt + s["dt_bias"]
    delta = torch.nn.functional.softplus(pre, threshold=700.0)
    h = s["init"].clone() if s["init"] is not None else x.new_zeros(Bt, E, N)
    train = mode == "train"
    kept = x.new_empty(L + 1, Bt, E, N) if train else None
    ys = torch.empty_like(x)
    grouped = lambda m, t: m[:, t].repeat_interleave(each, 1)  # noqa: E731
    for t in range(L):
        if train:
            kept[t] = h
        d = delta[:, t, :, None]
        h = torch.exp(d * A) * h + d * grouped(B, t) * x[:, t, :, None]
        ys[:, t] = (h * grouped(C, t)).sum(-1) + D * x[:, t]
    if train:
        kept[L] = h
    gate = torch.nn.functional.silu(z) if z is not None else torch.ones_like(x)
    y = ys * gate
    if mode == "step":
        return {"y": y[:, 0], "state": h}
    out = {"y": y, "final": h}
    if not train:
        return out
    dys = s["dy"] * gate
    if z is not None:
        sg = torch.sigmoid(z)
        out["dz"] = s["dy"] * ys * (sg + z * sg * (1 - sg))
    dx, ddelta, dB, dC = D * dys, torch.zeros_like(x), torch.zeros_like(B), torch.zeros_like(C)
    dA, g = torch.zeros_like(A), torch.zeros_like(h)
    for t in reversed(range(L)):
        d, Bt_, u = delta[:, t, :, None], grouped(B, t), x[:, t, :, None]
        g = g + dys[:, t, :, None] * grouped(C, t)
        a = torch.exp(d * A)
        dC[:, t] = (kept[t + 1] * dys[:, t, :, None]).unflatten(1, (G, each)).sum(2)
        dB[:, t] = (g * d * u).unflatten(1, (G, each)).sum(2)
        dx[:, t] += (g * Bt_ * d).sum(-1)
        back = g * a * kept[t]
        ddelta[:, t] = (g * Bt_ * u + back * A).sum(-1)
        dA += (back * d).sum(0)
        g = g * a
    ddt = ddelta * torch.sigmoid(pre)
    out.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dys * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))
    if s["init"] is not None:
        out["dinit"] = g
    return out


def _exact_norm(s):
    c = s["case"]
    train = c["mode"] == "train"
    x = s["x"]
    out = {}
    if s["residual"] is not None:
        out["sum"] = x + s["residual"]
        # the norm's input is the stream as it is kept, in its own type
        x = out["sum"].to(_type(c["residual"])).double()
    leaves = [v.clone().requires_grad_(train) if v is not None else None for v in (x, s["z"], s["weight"], s["bias"])]
    x, z, w, b = leaves
    u = x if z is None else x * torch.nn.functional.silu(z)
    D = c["width"]
    m = 0.0 if c["rms"] else u.sum(-1, keepdim=True) / D
    var = ((u - m) ** 2).sum(-1, keepdim=True) / D
    y = (u - m) / torch.sqrt(var + EPS) * w
    y = y if b is None else y + b
    out["y"] = y.detach()
    if not train:
        return out
    names = [("dx", x), ("dz", z), ("dweight", w), ("dbias", b)]
    got = torch.autograd.grad(y, [v for _, v in names if v is not None], s["dy"])
    out.update(zip([k for k, v in names if v is not None], got))
    if s["residual"] is not None:
        out["dx"] = out["dx"] + s["dresidual"]
        out["dresidual"] = out["dx"]
    return out
