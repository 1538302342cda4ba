"""Runs the kernels of the recurrent block's operators on the CPU (cpu_build.py), as
cases.py does those of the state-space layers. Usage:
cases_blocks.py LIBRARY [recurrence | dropout | block ...]."""
import ctypes
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import cases as K  # noqa: E402  (loads the library of the first argument)
import block_refs as B  # noqa: E402
import layer_refs as R  # noqa: E402

from structured_state_space_ssd_amd import _native  # noqa: E402

BF, F32, ptr, code, ok, every_way = K.BF, K.F32, K.ptr, K.code, K.ok, K.every_way
lib = K.lib
for _name, (_res, _args) in _native.BLOCK_SIGNATURES.items():
    getattr(lib, _name).restype, getattr(lib, _name).argtypes = _res, _args


def scratch(m, size):
    """Address and size of a workspace; none where none is needed."""
    return (ptr(m.bytes(size)), size) if size else (None, 0)


# ---- recurrence -------------------------------------------------------------------------

# (batch, tokens, channels): one token, parts of a strand and of a wavefront's tokens, whole
# and ragged tiles of 1 to 16 wavefronts, odd channels around the 32 of a workgroup, plans
# with segments (few channels and several tiles)
SIZES = [(1, 1, 1), (2, 7, 3), (1, 8, 32), (3, 31, 33), (1, 32, 64), (2, 33, 31), (1, 100, 34), (1, 520, 5),
         (2, 700, 33), (1, 1100, 2)]


def recurrence(size, dtype, gated, gate, pad, ends, cu=None, keep=True):
    Bt, L, E = size
    g = torch.Generator().manual_seed(sum(size))
    r = lambda *s, dt=dtype, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt)  # noqa: E731
    a = dict(x=r(Bt, L, E + pad)[..., pad:], r=r(Bt, L, E + pad)[..., :E], i=None, decay=None)
    if gated:
        a["i"], a["decay"] = r(Bt, L, E), r(E, dt=F32, sc=2.0, off=-4.0)
    else:
        a["r"] = -a["r"].abs()
    a["z"] = r(Bt, L, 2 * E)[..., E:] if gate else None
    init = r(Bt, E, dt=F32) if ends and cu is None else None
    nseq = 0 if cu is None else len(cu) - 1
    dy, dfinal = r(Bt, L, E), r(nseq or Bt, E, dt=F32) if ends else None
    want = B.recurrence(*a.values(), init, 8.0, cu, (dy, dfinal))
    keeps = -(-L // B.KEEP)

    def inputs(m):
        p = {k: m.put(v) for k, v in a.items()}
        st = []
        for k in ("x", "r", "i", "z"):
            st += (0, 0) if p[k] is None else p[k].stride()[:2]
        pc = None if cu is None else m.put(torch.tensor(cu, dtype=torch.int32))
        return p, [ptr(p[k]) for k in ("x", "r", "i", "decay")] + [8.0, ptr(p["z"])], pc, ctypes.byref(
            _native.SsdRecurrenceStrides(*st))

    def forward(m):
        p, args, pc, st = inputs(m)
        o = dict(y=m.new((Bt, L, E), dtype), final=m.new((nseq or Bt, E)), states=m.new((Bt, keeps, E)))
        ws = scratch(m, lib.ssd_recurrence_forward_workspace_size(Bt, L, E, int(nseq > 0), code(dtype)))
        ok(lib.ssd_recurrence_forward(*args, Bt, L, E, code(dtype), ptr(m.put(init)), ptr(pc), nseq, ptr(o["y"]),
                                      ptr(o["final"]), ptr(o["states"]), *ws, st, None), "forward")
        return o

    name = (size, str(dtype), gated, gate, pad, cu)
    got = every_way(name, forward)
    kept = got["states"]

    def backward(m):
        p, args, pc, st = inputs(m)
        o = dict(dx=m.new((Bt, L, E), dtype), dr=m.new((Bt, L, E), dtype), di=m.new((Bt, L, E), dtype) if gated else None,
                 ddecay=m.new((E,)) if gated else None, dz=m.new((Bt, L, E), dtype) if gate else None,
                 dinit=m.new((Bt, E)) if init is not None else None)
        ws = scratch(m, lib.ssd_recurrence_backward_workspace_size(Bt, L, E, int(nseq > 0), int(keep), code(dtype)))
        ok(lib.ssd_recurrence_backward(*args, ptr(m.put(init)), ptr(pc), nseq, ptr(m.put(kept)) if keep else None,
                                       ptr(m.put(dy)), ptr(m.put(dfinal)), Bt, L, E, code(dtype),
                                       *map(ptr, o.values()), *ws, st, None), "backward")
        return o

    def step(m):
        p, args, _, _ = inputs(m)
        state, y = m.put(init), m.new((Bt, E), dtype)
        st = []
        for k in ("x", "r", "i", "z"):
            st += (0, 0) if p[k] is None else (p[k].stride(0), -1)
        ok(lib.ssd_recurrence_step(ptr(state), *args, Bt, E, code(dtype), ptr(y),
                                   ctypes.byref(_native.SsdRecurrenceStrides(*st)), None), "step")
        return dict(y=y, state=state)

    got.update(every_way(name, backward))
    for k, v in got.items():
        if v is not None:
            R.check((name, k), v, want[k], want[k + "_err"], 1.0)
    if init is not None:
        one = every_way(name, step)
        R.check((name, "step"), one["y"], want["y"][:, 0], want["y_err"][:, 0], 1.0)
        first = B.recurrence(*[v if v is None or v.dim() == 1 else v[:, :1] for v in a.values()], init)
        R.check((name, "state"), one["state"], first["final"], first["final_err"], 1.0)


def bad_offsets(cu):
    """Offsets that no sequence has: nothing is read or written outside (what comes is not said)."""
    L, E, nseq = 100, 5, len(cu) - 1
    x = torch.randn(1, L, E)

    def run(m):
        px, pr, pd, pc = m.put(x), m.put(-x.abs()), m.put(x), m.put(torch.tensor(cu, dtype=torch.int32))
        o = dict(y=m.new((1, L, E)), final=m.new((nseq, E)), states=m.new((1, 7, E)), dx=m.new((1, L, E)),
                 dr=m.new((1, L, E)))
        ws = scratch(m, lib.ssd_recurrence_forward_workspace_size(1, L, E, 1, 0))
        ok(lib.ssd_recurrence_forward(ptr(px), ptr(pr), None, None, 8.0, None, 1, L, E, 0, None, ptr(pc), nseq,
                                      ptr(o["y"]), ptr(o["final"]), ptr(o["states"]), *ws, None, None),
           "forward")
        ws = scratch(m, lib.ssd_recurrence_backward_workspace_size(1, L, E, 1, 1, 0))
        ok(lib.ssd_recurrence_backward(ptr(px), ptr(pr), None, None, 8.0, None, None, ptr(pc), nseq, ptr(o["states"]),
                                       ptr(pd), ptr(m.put(torch.randn(nseq, E, generator=torch.Generator().manual_seed(1)))),
                                       1, L, E, 0, ptr(o["dx"]), ptr(o["dr"]), None, None, None, None, *ws,
                                       None, None), "backward")
        return o

    every_way(cu, run)


def growth(L, rate, dtype, cu=None):
    """Log-decays above 0 over tiles of zero inputs, whose products pass float32: a state of zero
    stays zero. Inputs are at the last tokens only, gradients of y at the first."""
    E, few = 5, 6
    g = torch.Generator().manual_seed(L)
    x, r, dy = (torch.zeros(1, L, E, dtype=dtype) for _ in range(3))
    r.fill_(rate)
    x[:, -few:], dy[:, :few] = torch.randn(1, few, E, generator=g).to(dtype), torch.randn(1, few, E, generator=g).to(dtype)
    nseq = 0 if cu is None else len(cu) - 1
    want = B.recurrence(x, r, cu=cu, grads=(dy, None))

    def run(m):
        px, pr, pd, pc = m.put(x), m.put(r), m.put(dy), None if cu is None else m.put(torch.tensor(cu, dtype=torch.int32))
        o = dict(y=m.new((1, L, E), dtype), final=m.new((nseq or 1, E)), dx=m.new((1, L, E), dtype), dr=m.new((1, L, E), dtype))
        c = code(dtype)
        ws = scratch(m, lib.ssd_recurrence_forward_workspace_size(1, L, E, int(nseq > 0), c))
        ok(lib.ssd_recurrence_forward(ptr(px), ptr(pr), None, None, 8.0, None, 1, L, E, c, None, ptr(pc), nseq, ptr(o["y"]),
                                      ptr(o["final"]), None, *ws, None, None), "forward")
        ws = scratch(m, lib.ssd_recurrence_backward_workspace_size(1, L, E, int(nseq > 0), 0, c))
        ok(lib.ssd_recurrence_backward(ptr(px), ptr(pr), None, None, 8.0, None, None, ptr(pc), nseq, None, ptr(pd), None,
                                       1, L, E, c, ptr(o["dx"]), ptr(o["dr"]), None, None, None, None, *ws, None, None),
           "backward")
        return o

    for k, v in every_way((L, rate, cu), run).items():
        R.check((L, rate, str(dtype), cu, k), v, want[k], want[k + "_err"], 1.0)


def run_growth():
    for L, rate in ((100, 1.0), (520, 1.0), (1100, 0.5), (2500, 0.5), (300, 8.0)):
        for dtype in (BF, F32):
            for cu in (None, [0, 3, L]):
                print("growth", L, rate, dtype, cu, flush=True)
                growth(L, rate, dtype, cu)


def run_recurrence():
    for size in SIZES:
        for args in ((BF, True, True, 3, True), (F32, True, False, 0, False), (BF, False, False, 0, True),
                     (F32, False, True, 1, True)):
            print("recurrence", size, *args, flush=True)
            recurrence(size, *args, keep=args[0] is BF)
    # sequences inside strands, across wavefronts, tiles and segments, empty ones, one of one token
    for L, cu in ((40, [0, 40]), (40, [0, 0, 1, 2, 2, 15, 31, 40, 40]), (700, [0, 3, 300, 300, 301, 511, 700]),
                  (300, [7, 9, 64, 200]),
                  (1100, [0, 64, 1000, 1100]), (1030, list(range(0, 1031, 103)))):
        for args in ((BF, True, True, 3, True), (F32, False, False, 0, True), (F32, True, False, 0, False)):
            print("recurrence packed", cu, *args, flush=True)
            recurrence((1, L, 5), *args, cu=cu, keep=args[0] is BF)
    for cu in ([0, 30], [5, 20, 100], [0, -7, 1 << 30, 100], [100, 0, 100], [-(1 << 31), (1 << 31) - 1], [0, 190, 80, -3]):
        print("recurrence packed, not offsets:", cu, flush=True)
        bad_offsets(cu)


# ---- dropout ------------------------------------------------------------------------------

def dropout(rows, D, dtype, pad, p, on_gpu):
    g = torch.Generator().manual_seed(rows + D)
    x, rng = torch.randn(rows, D + pad, generator=g).to(dtype)[:, pad:], ((1 << 63) + 12345, (5 << 32) + 7)

    def run(m):
        px, y = m.put(x), m.new((rows, D), dtype)
        state = m.new((2,), torch.int64, fill=0)
        state[0], state[1] = rng[0] - (1 << 64), rng[1]
        r = _native.SsdRandom(p, 1, 2, ptr(state)) if on_gpu else _native.SsdRandom(p, *rng, None)
        ok(lib.ssd_dropout(ptr(px), px.stride(0), rows, D, ctypes.byref(r), code(dtype), ptr(y), None), "dropout")
        return dict(y=y)

    want = B.dropped(x, p, rng)
    R.check((rows, D, p), every_way((rows, D, p), run)["y"], want, want.abs(), 3)


def run_dropout():
    for rows, D in ((1, 1), (3, 7), (40, 8), (5, 9), (300, 33), (7, 1000), (1, 16390)):
        for dtype, pad, p, on_gpu in ((BF, 3, 0.1, False), (F32, 0, 0.5, True), (BF, 0, 1.0, False), (F32, 1, 0.0, False)):
            print("dropout", rows, D, dtype, pad, p, flush=True)
            dropout(rows, D, dtype, pad, p, on_gpu)


# ---- block norm -----------------------------------------------------------------------------

# every lane count of short rows, one, two and four vectors to a lane of long ones, rows past
# the groups of a workgroup, and some of the last round of several rows to a workgroup
BLOCK = [(1, 1), (3, 7), (300, 8), (70, 16), (65, 40), (9, 250), (5, 511), (3, 513), (7, 1300), (2, 2000), (4, 2563),
         (2, 4097), (1, 5200), (1, 6200), (1, 8191), (1, 8192)]


def block(rows, D, dtype, stream, rms, post, pre, bias, scale, gate, p, pad, skip):
    g = torch.Generator().manual_seed(rows + D)
    r = lambda *s, dt=dtype, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt)  # noqa: E731
    x, res = r(rows, D + pad, off=0.5)[:, pad:], r(rows, D, dt=stream)
    par = dict(weight=r(D, dt=F32, off=1.0) if pre else None, bias=r(D, dt=F32) if pre and bias else None,
               post_weight=r(D, dt=F32, off=1.0) if post else None, post_bias=r(D, dt=F32) if post and bias else None,
               scale=r(D, dt=F32) if scale else None)
    z = r(rows, D + pad)[:, :D] if gate else None
    dy, dsum = r(rows, D) if pre else None, r(rows, D, dt=stream) if skip else None
    alpha, beta, eps, rng = 1.25, -0.75, 1e-5, (77, 9)
    ref = B.Block(x, res, *par.values(), z, alpha, beta, p, rng, eps, rms)

    def options(m):
        kept = {k: m.put(v) for k, v in par.items()}
        rnd = ctypes.byref(_native.SsdRandom(p, *rng, None)) if p else None
        return kept, ctypes.byref(_native.SsdBlock(*map(ptr, kept.values()), alpha, beta, int(rms), eps)), rnd

    def forward(m):
        keep, opt, rnd = options(m)
        px, pr, pz = m.put(x), m.put(res), m.put(z)
        o = dict(y=m.new((rows, D), dtype) if pre else None, sum=m.new((rows, D), stream),
                 mean=m.new((rows,)) if pre and not rms else None, rstd=m.new((rows,)) if pre else None,
                 post_mean=m.new((rows,)) if post and not rms else None, post_rstd=m.new((rows,)) if post else None)
        ok(lib.ssd_block_norm_forward(ptr(px), px.stride(0), ptr(pr), code(stream), ptr(pz), 0 if z is None else pz.stride(0),
                                      opt, rnd, rows, D, code(dtype), *map(ptr, o.values()), None), "forward")
        return o

    name = (rows, D, str(dtype), str(stream), rms, post, pre, bias, scale, gate, p)
    f = every_way(name, forward)
    # one norm takes 122 roundings (test_gpu_norm.py), the gate 8 + 2 |z|, the products and sums 6
    kz = 0 if z is None else 8 + 2 * float(z.abs().max())
    R.check((name, "sum"), f["sum"], ref.total, ref.total_mag, 128 + kz)
    if pre:
        y, mag = ref.y(f["sum"])
        R.check((name, "y"), f["y"], y, mag, 122)

    def backward(m):
        keep, opt, rnd = options(m)
        pd, ps, px, pt, pz = m.put(dy), m.put(dsum), m.put(x), m.put(f["sum"]), m.put(z)
        st = [m.put(f[k]) for k in ("mean", "rstd", "post_mean", "post_rstd")]
        o = dict(dx=m.new((rows, D), dtype), dresidual=m.new((rows, D), stream), dz=m.new((rows, D), dtype) if gate else None)
        for k, v in par.items():
            o["d" + k] = m.new((D,)) if v is not None else None
        ws = scratch(m, lib.ssd_block_norm_backward_workspace_size(rows, D, code(dtype)))
        ok(lib.ssd_block_norm_backward(ptr(pd), ptr(ps), ptr(px), px.stride(0), ptr(pt), code(stream), ptr(pz),
                                       0 if z is None else pz.stride(0), opt, rnd, *map(ptr, st), rows, D, code(dtype),
                                       *map(ptr, o.values()), *ws, None), "backward")
        return o

    got = every_way(name, backward)
    want, mag = ref.grads(dy, dsum, f["sum"])
    for k, t in got.items():
        if t is not None:  # two norms and their gradients, the gate twice, sums over the rows
            many = rows if k not in ("dx", "dresidual", "dz") else 0
            R.check((name, k), t, want[k], mag[k], 4 * 122 + 2 * kz + 16 + many)


def run_block():
    for rows, D in BLOCK:
        for args in ((BF, F32, True, True, True, False, True, False, 0.3, 3, True),
                     (F32, F32, False, True, True, True, True, True, 0.1, 1, True),
                     (BF, BF, False, True, True, True, False, True, 0.0, 0, False),
                     (BF, F32, False, False, True, True, True, True, 0.5, 0, True),
                     (F32, F32, True, True, False, False, False, False, 0.0, 2, True)):
            print("block", rows, D, *args, flush=True)
            block(rows, D, *args)


def dropped(rows, D, dtype, stream, rms, post, bias, gate, p, bad):
    """What x (without a norm in front) and the gate hold where an element is dropped reaches no
    result and no gradient: the same bits as with zeros there."""
    g = torch.Generator().manual_seed(rows + D)
    r = lambda *s, dt=F32, off=0.0: (torch.randn(*s, generator=g) + off).to(dt)  # noqa: E731
    rng, kept = (5, 6), B.kept(rows, D, p, 5, 6)
    x, res, dy, dsum = r(rows, D, dt=dtype), r(rows, D, dt=stream), r(rows, D, dt=dtype), r(rows, D, dt=stream)
    par = [r(D, off=1.0), r(D) if bias else None, r(D, off=1.0) if post else None, r(D) if post and bias else None, r(D)]
    z = r(rows, D, dt=dtype) if gate else None

    def run(fill):
        tx = x if post else x.masked_fill(~kept, fill)
        tz = z.masked_fill(~kept, fill) if gate else None

        def both(m):
            put = [m.put(t) for t in par]
            opt = ctypes.byref(_native.SsdBlock(*map(ptr, put), 1.25, -0.75, int(rms), 1e-5))
            rnd = ctypes.byref(_native.SsdRandom(p, *rng, None))
            px, pr, pz, pd, ps = m.put(tx), m.put(res), m.put(tz), m.put(dy), m.put(dsum)
            o = dict(y=m.new((rows, D), dtype), sum=m.new((rows, D), stream), mean=None if rms else m.new((rows,)),
                     rstd=m.new((rows,)), post_mean=m.new((rows,)) if post and not rms else None,
                     post_rstd=m.new((rows,)) if post else None)
            stats = [ptr(o[k]) for k in ("mean", "rstd", "post_mean", "post_rstd")]
            ok(lib.ssd_block_norm_forward(ptr(px), D, ptr(pr), code(stream), ptr(pz), D, opt, rnd, rows, D, code(dtype),
                                          ptr(o["y"]), ptr(o["sum"]), *stats, None), "forward")
            q = dict(dx=m.new((rows, D), dtype), dresidual=m.new((rows, D), stream), dz=m.new((rows, D), dtype) if gate else None)
            for k, t in zip(("dweight", "dbias", "dpost_weight", "dpost_bias", "dscale"), par):
                q[k] = None if t is None else m.new((D,))
            ws = scratch(m, lib.ssd_block_norm_backward_workspace_size(rows, D, code(dtype)))
            ok(lib.ssd_block_norm_backward(ptr(pd), ptr(ps), ptr(px), D, ptr(o["sum"]), code(stream), ptr(pz), D, opt, rnd,
                                           *stats, rows, D, code(dtype), *map(ptr, q.values()), *ws, None), "backward")
            return {**o, **q}

        return every_way((rows, D, fill), both)

    want, got = run(0.0), run(bad)
    for k, t in got.items():
        assert t is None or torch.equal(t, want[k]), (k, "what is dropped matters")
        assert t is None or bool(t.isfinite().all()), k


def run_dropped():
    for rows, D in ((5, 9), (3, 513), (2, 2563), (1, 8192)):
        for args in ((BF, F32, True, False, False, False, 0.5), (BF, F32, False, True, True, True, 0.3),
                     (F32, F32, False, False, True, True, 0.5), (BF, BF, True, False, False, True, 0.9),
                     (F32, F32, True, False, False, False, 1.0), (F32, F32, True, True, False, True, 0.1)):
            for bad in (float("inf"), float("nan")):
                print("dropped", rows, D, *args, bad, flush=True)
                dropped(rows, D, *args, bad)


if __name__ == "__main__":
    torch.set_num_threads(1)
    for which in sys.argv[2:] or ("recurrence", "dropout", "block"):
        globals()["run_" + which]()
    print("all cases done")
