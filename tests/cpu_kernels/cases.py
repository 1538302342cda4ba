"""Runs the layers' kernels on the CPU (cpu_build.py) over state sizes, widths and
plans that reach each of their loops, every tensor and workspace between
unmapped pages, and compares with the plain 64-bit forms. Usage:
cases.py LIBRARY [selective | conv | norm ...]. Prints every case before it
runs; an access out of range ends the process there."""
import ctypes
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), os.path.dirname(os.path.dirname(HERE))]
import layer_refs as R  # noqa: E402

from structured_state_space_ssd_amd import _native  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
lib = ctypes.CDLL(sys.argv[1])
for _name, (_res, _args) in _native.SIGNATURES.items():
    if any(k in _name for k in ("conv", "selective", "norm")):
        getattr(lib, _name).restype, getattr(lib, _name).argtypes = _res, _args
lib.cpu_alloc.restype, lib.cpu_alloc.argtypes = ctypes.c_void_p, [ctypes.c_size_t, ctypes.c_int]
lib.cpu_free.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]


class Memory:
    """Tensors against the page behind them (right) or the one in front."""

    def __init__(self, right):
        self.right, self.held, self.tails = right, [], []

    def new(self, shape, dtype=F32, stride=None, fill=float("nan")):
        """A tensor in memory of its own, which ends with its last element."""
        shape = tuple(shape)
        if stride is None:
            stride = torch.empty(shape, device="meta").stride()
        count = 1 + sum((n - 1) * s for n, s in zip(shape, stride))
        size = count * torch.tensor([], dtype=dtype).element_size()
        at = lib.cpu_alloc(size, self.right)
        self.held.append((at, size))
        flat = torch.frombuffer((ctypes.c_char * size).from_address(at), dtype=dtype)
        flat.fill_(fill if dtype.is_floating_point or fill == fill else -1)
        return flat.as_strided(shape, stride)

    def put(self, t):
        return None if t is None else self.new(t.shape, t.dtype, t.stride()).copy_(t)

    def bytes(self, size):
        """A workspace: 256-byte aligned, so up to 255 bytes short of the page; nothing
        may be written to those either."""
        whole = self.new(((size + 255) // 256 * 256,), torch.uint8, fill=0xff)
        self.tails.append(whole[size:])
        return whole[:size]

    def free(self):
        for tail in self.tails:
            assert bool((tail == 0xff).all()), "written past the workspace"
        for at, size in self.held:
            lib.cpu_free(at, size, self.right)
        self.held = []


def ptr(t):
    return None if t is None else t.data_ptr()


def code(dtype):
    return _native.SSD_BF16 if dtype == BF else _native.SSD_F32


def ok(rc, what):
    assert rc == 0, (what, rc)


def same(a, b, what):
    """The same bits, whatever order the lanes ran in."""
    for k in a:
        assert a[k] is None or torch.equal(a[k], b[k]), (what, k, "depends on the lanes' order")


def every_way(name, run):
    """run(memory) with the pages on either side and the lanes in three orders."""
    first = None
    for right, order in ((1, 0), (0, 1), (1, 7)):
        lib.cpu_order(order)
        m = Memory(right)
        out = {k: None if v is None else v.clone() for k, v in run(m).items()}
        m.free()
        if first is None:
            first = out
        else:
            same(first, out, name)
    return first


# ---- selective scan ---------------------------------------------------------------

# (batch, tokens, channels, states, groups): every kernel state size at and below it,
# ragged channels, one token, tiles with a last one part full, one piece and segments
# (the plan cuts what leaves CUs without work: 4 tiles and more here), tokens that fill
# the last tile, past which the next ones' B and C are fetched all the same, and batches
# just past the CUs, of which only the rest is cut
SELECTIVE = [(1, 1, 1, 1, 1), (2, 9, 5, 3, 1), (1, 40, 300, 4, 1), (1, 37, 130, 7, 2), (2, 70, 70, 8, 1),
             (1, 33, 70, 13, 2), (1, 150, 66, 16, 1), (1, 70, 34, 24, 2), (1, 140, 65, 32, 1),
             (1, 32, 66, 16, 1), (1, 64, 20, 64, 1),
             (1, 40, 20, 64, 1), (1, 33, 66, 50, 2), (1, 140, 9, 64, 1), (257, 20, 4, 3, 1), (1, 330, 6, 3, 2)]


def selective(size, dtype, gate, pad, soft, D=True, init=True):
    Bt, L, E, N, G = size
    g = torch.Generator().manual_seed(sum(size))
    r = lambda *s, dt=dtype, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt)  # noqa: E731
    a = dict(x=r(Bt, L, E + pad)[..., pad:], dt=r(Bt, L, E, sc=0.5) if soft else r(Bt, L, E).abs() * 0.05,
             A=-torch.exp(torch.rand(E, N, generator=g) * 2.77))
    bc = r(Bt, L, pad + 2 * G * N, sc=N ** -0.5)
    a["B"] = bc[..., pad:pad + G * N].unflatten(-1, (G, N))
    a["C"] = bc[..., pad + G * N:].unflatten(-1, (G, N))
    a["D"] = r(E, dt=F32) if D else None
    a["z"] = r(Bt, L, E + pad)[..., :E] if gate else None
    a["init"] = r(Bt, E, N, dt=F32) if init else None
    a["bias"] = r(E, dt=F32, off=-3.0) if soft else None
    limit = (0.01, 0.3) if soft else None
    dy, dfinal = r(Bt, L, E), r(Bt, E, N, dt=F32) if init else None
    want = R.selective(*a.values(), soft, limit, (dy, dfinal))

    def inputs(m):
        p = {k: m.put(v) for k, v in a.items()}
        st = []
        for k in ("x", "dt", "z", "B", "C"):
            st += (0, 0) if p[k] is None else p[k].stride()[:2]
        strides = ctypes.byref(_native.SsdSelectiveStrides(*st))
        opts = _native.SsdOptions(ptr(p["bias"]), int(soft), int(soft), 0.01, 0.3, 0) if soft else None
        args = [ptr(p[k]) for k in ("x", "dt", "A", "B", "C", "D", "z")]
        return p, args, strides, None if opts is None else ctypes.byref(opts)

    def forward(m):
        p, args, strides, opts = inputs(m)
        y, final = m.new((Bt, L, E), dtype), m.new((Bt, E, N))
        ws = m.bytes(lib.ssd_selective_forward_workspace_size(Bt, L, E, G, N, code(dtype)))
        ok(lib.ssd_selective_forward(*args, Bt, L, E, G, N, code(dtype), ptr(p["init"]), ptr(y), ptr(final), ptr(ws),
                                     ws.numel(), strides, opts, None), "forward")
        return dict(y=y, final=final)

    def backward(m):
        p, args, strides, opts = inputs(m)
        o = dict(dx=m.new((Bt, L, E), dtype), ddt=m.new((Bt, L, E), dtype), dA=m.new((E, N)),
                 dB=m.new((Bt, L, G, N), dtype), dC=m.new((Bt, L, G, N), dtype), dD=m.new((E,)),
                 dz=m.new((Bt, L, E), dtype) if gate else None, dinit=m.new((Bt, E, N)),
                 ddt_bias=m.new((E,)) if soft else None)
        dys, df = m.put(dy), m.put(dfinal)
        ws = m.bytes(lib.ssd_selective_backward_workspace_size(Bt, L, E, G, N, code(dtype)))
        ok(lib.ssd_selective_backward(*args, ptr(p["init"]), ptr(dys), ptr(df), Bt, L, E, G, N, code(dtype),
                                      *map(ptr, o.values()), ptr(ws), ws.numel(), strides, opts, None), "backward")
        return o

    def step(m):
        p, args, _, opts = inputs(m)
        state = m.put(a["init"])
        y = m.new((Bt, E), dtype)
        st = []
        for k in ("x", "dt", "z", "B", "C"):
            st += (0, 0) if p[k] is None else (p[k].stride(0), -1)
        ok(lib.ssd_selective_step(ptr(state), *args, Bt, E, G, N, code(dtype), ptr(y),
                                  ctypes.byref(_native.SsdSelectiveStrides(*st)), opts, None), "step")
        return dict(y=y, state=state)

    name = (size, str(dtype), gate, pad)
    got = {**every_way(name, forward), **every_way(name, backward)}
    for k, v in got.items():
        if v is not None:
            R.check((name, k), v, want[k], want[k + "_err"], 1.0)
    if init:
        one = every_way(name, step)
        R.check((name, "step"), one["y"], want["y"][:, 0], want["y_err"][:, 0], 1.0)


def run_selective():
    for size in SELECTIVE:
        for dtype, gate, pad, soft in ((BF, True, 5, True), (BF, False, 0, False), (F32, True, 3, True)):
            print("selective", size, dtype, gate, pad, flush=True)
            selective(size, dtype, gate, pad, soft, D=soft, init=gate or size[1] < 50)


# ---- convolution --------------------------------------------------------------------

CONV = [(1, 1, 1, None), (2, 1, 9, None), (1, 3, 8, None), (3, 17, 33, None), (1, 40, 25, (17, 3, 5)),
        (2, 9, 1030, (1000, 21, 9)), (1, 16700, 2, None)]


def conv(Bt, L, K, split, W, dtype, act, pad, ends, bias):
    g = torch.Generator().manual_seed(L + K + W)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    x, w, b = r(Bt, L, K + pad)[..., pad:], r(K, W, dt=F32), r(K, dt=F32) if bias else None
    init, dfinal = (r(Bt, W - 1, K), r(Bt, W - 1, K)) if ends else (None, None)
    parts = split or (K,)
    dy = [r(Bt, L, k) for k in parts]
    arr, n = ((ctypes.c_int * len(split))(*split), len(split)) if split else (None, 0)
    table = lambda ts: (ctypes.c_void_p * len(ts))(*map(ptr, ts))  # noqa: E731

    def forward(m):
        px, pw, pb, pi = m.put(x), m.put(w), m.put(b), m.put(init)
        ys, final = [m.new((Bt, L, k), dtype) for k in parts], m.new((Bt, W - 1, K), dtype)
        ok(lib.ssd_conv_forward(ptr(px), px.stride(0), px.stride(1), ptr(pw), ptr(pb), ptr(pi), None, 0, Bt, L, K, W,
                                act, code(dtype), arr, n, table(ys), ptr(final), None), "forward")
        return dict(y=torch.cat(ys, -1), final=final)

    def backward(m):
        px, pw, pb, pi = m.put(x), m.put(w), m.put(b), m.put(init)
        dys, pf = [m.put(t) for t in dy], m.put(dfinal)
        o = dict(dx=m.new((Bt, L, K), dtype), dweight=m.new((K, W)), dbias=m.new((K,)) if bias else None,
                 dinit=m.new((Bt, W - 1, K), dtype) if ends else None)
        ws = m.bytes(lib.ssd_conv_backward_workspace_size(Bt, L, K, W, code(dtype)))
        ok(lib.ssd_conv_backward(ptr(px), px.stride(0), px.stride(1), ptr(pw), ptr(pb), ptr(pi), arr, n, table(dys),
                                 ptr(pf), Bt, L, K, W, act, code(dtype), *map(ptr, o.values()), ptr(ws), ws.numel(),
                                 None), "backward")
        return o

    def step(m):
        px, pw, pb, state = m.put(x[:, 0]), m.put(w), m.put(b), m.put(init)
        ys = [m.new((Bt, k), dtype) for k in parts]
        ok(lib.ssd_conv_step(ptr(state), ptr(px), px.stride(0), ptr(pw), ptr(pb), Bt, K, W, act, code(dtype), arr, n,
                             table(ys), None), "step")
        return dict(y=torch.cat(ys, -1), state=state)

    name = (Bt, L, K, split, W, str(dtype))
    got = every_way(name, forward)
    v, y, final, mag = R.conv(x, w, b, act, init)
    R.check((name, "y"), got["y"], y, 1.1 * (W + 1) * mag + (y.abs() * (8 + 2 * v.abs()) if act else 0), 1.0)
    assert torch.equal(got["final"].double(), final)
    got = every_way(name, backward)
    want, wmag = R.conv_grads(x, w, b, act, torch.cat(dy, -1), init, dfinal)
    for k, t in got.items():
        if t is not None:  # counted in test_gpu_conv.py
            R.check((name, k), t, want[k], wmag[k], W + 14 + (W + 1) * float(mag.max()) + (Bt * L if k[1] in "wb" else 0))
    if ends:
        one = every_way(name, step)
        assert torch.equal(one["y"], every_way(name, forward)["y"][:, 0])
        xs = torch.cat([init, x[:, :1]], 1)
        assert torch.equal(one["state"], xs[:, 1:])


def packed(cu, W, dtype, bad=False):
    """Packed sequences; `bad`: offsets that no sequence has read and write nothing
    outside (what they give is not said)."""
    L, K = 40, 21
    g = torch.Generator().manual_seed(W)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    x, w, b = r(1, L, K + 2)[..., 2:], r(K, W, dt=F32), r(K, dt=F32)

    def forward(m):
        px, pw, pb, pc = m.put(x), m.put(w), m.put(b), m.put(torch.tensor(cu, dtype=torch.int32))
        y, final = m.new((1, L, K), dtype), m.new((len(cu) - 1, W - 1, K), dtype)
        ok(lib.ssd_conv_forward(ptr(px), px.stride(0), px.stride(1), ptr(pw), ptr(pb), None, ptr(pc), len(cu) - 1, 1,
                                L, K, W, 1, code(dtype), None, 0, (ctypes.c_void_p * 1)(ptr(y)), ptr(final), None),
           "packed")
        return dict(y=y, final=final)

    got = every_way(cu, forward)
    if not bad:
        v, y, final, mag = R.conv(x, w, b, True, None, cu)
        R.check((cu, "y"), got["y"], y, 1.1 * (W + 1) * mag + y.abs() * (8 + 2 * v.abs()), 1.0)
        assert torch.equal(got["final"].double(), final)


def run_conv():
    for Bt, L, K, split in CONV:
        long = L > 1000  # more partial rows than one pass sums up
        for W, dtype, act, pad, ends, bias in ((4, BF, 1, 3, True, True), (3, F32, 0, 0, False, False),
                                               (2, F32, 1, 1, True, True))[2 if long else 0:]:
            print("conv", Bt, L, K, split, W, dtype, flush=True)
            conv(Bt, L, K, split, W, dtype, act, pad, ends, bias)
    for cu in ([0, 40], [0, 0, 1, 2, 2, 15, 31, 40], list(range(0, 41, 5))):
        print("packed", cu, flush=True)
        packed(cu, 4, BF)
        packed(cu, 2, F32)
    for cu in ([0, 30], [5, 20, 40], [0, -7, 1 << 30, 40], [40, 0, 40], [-(1 << 31), (1 << 31) - 1], [0, 90, 80, -3]):
        print("packed, not offsets:", cu, flush=True)
        packed(cu, 3, BF, bad=True)


# ---- norm ---------------------------------------------------------------------------

# every lane count of short rows, one and several vectors to a lane of long ones, rows
# past the groups of a workgroup
NORM = [(1, 1), (3, 7), (300, 8), (70, 16), (65, 40), (9, 100), (9, 250), (5, 511), (3, 513), (2, 2000),
        (2, 4097), (1, 8193), (1, 16384)]


def norm(rows, D, dtype, stream, gate, rms, bias, pad, skip):
    g = torch.Generator().manual_seed(rows + D)
    r = lambda *s, dt=dtype, off=0.0: (torch.randn(*s, generator=g) + off).to(dt)  # noqa: E731
    x, w, b = r(rows, D + pad, off=0.5)[:, pad:], r(D, dt=F32, off=1.0), r(D, dt=F32) if bias else None
    res = r(rows, D, dt=stream) if stream else None
    z = r(rows, D + pad)[:, :D] if gate else None
    dy, dres = r(rows, D), r(rows, D, dt=stream) if stream and skip else None
    eps, none = 1e-5, torch.empty(0)

    def forward(m):
        px, pw, pb, pr, pz = m.put(x), m.put(w), m.put(b), m.put(res), m.put(z)
        o = dict(y=m.new((rows, D), dtype), sum=None if res is None else m.new((rows, D), stream),
                 mean=None if rms else m.new((rows,)), rstd=m.new((rows,)))
        ok(lib.ssd_norm_forward(ptr(px), px.stride(0), ptr(pr), code(stream), ptr(pz), 0 if z is None else pz.stride(0),
                                ptr(pw), ptr(pb), rows, D, int(rms), eps, code(dtype), *map(ptr, o.values()), None),
           "forward")
        return o

    name = (rows, D, str(dtype), str(stream), gate, rms)
    f = every_way(name, forward)
    u = f["sum"] if stream else x

    def backward(m):
        pd, pu, pz, pw, pm, ps, pr = map(m.put, (dy, u, z, w, f["mean"], f["rstd"], dres))
        o = dict(dx=m.new((rows, D), dtype), dres=m.new((rows, D), stream) if stream else None,
                 dz=m.new((rows, D), dtype) if gate else None, dweight=m.new((D,)), dbias=m.new((D,)) if bias else None)
        ws = m.bytes(lib.ssd_norm_backward_workspace_size(rows, D, code(dtype), int(bias)))
        ok(lib.ssd_norm_backward(ptr(pd), ptr(pu), pu.stride(0), code(u.dtype), ptr(pz), 0 if z is None else pz.stride(0),
                                 ptr(pw), ptr(pm), ptr(ps), ptr(pr), rows, D, code(dtype), *map(ptr, o.values()), ptr(ws),
                                 ws.numel(), None), "backward")
        return o

    want, _, _, mag = R.norm(u, w, b, rms, eps, z)
    ops = 122 + (0 if z is None else 2 * (8 + 2 * float(z.abs().max())))  # counted in test_gpu_norm.py
    R.check((name, "y"), f["y"], want, mag, ops)
    got = every_way(name, backward)
    want, mag = R.norm_grads(dy, u, w, rms, eps, z, dres)
    want["dres"], mag["dres"] = want["dx"], mag["dx"]
    for k, t in got.items():
        if t is not None:
            R.check((name, k), t, want[k], mag[k], 2 * ops + (rows if k in ("dweight", "dbias") else 0))


def run_norm():
    for rows, D in NORM:
        for args in ((BF, F32, False, False, True, 3, True), (BF, None, True, True, False, 5, False),
                     (F32, F32, False, True, True, 0, False), (F32, None, True, False, True, 1, False),
                     (BF, BF, False, True, False, 0, False)):
            print("norm", rows, D, *args, flush=True)
            norm(rows, D, *args)


if __name__ == "__main__":
    torch.set_num_threads(1)
    for which in sys.argv[2:] or ("selective", "conv", "norm"):
        globals()["run_" + which]()
    print("all cases done")
