"""The convolution, the scans and the normalisation run together as a block of a
model runs them: a prompt, the tokens after it and a training step. Each
operator is checked against its plain 64-bit form on the inputs that it got, so
the tolerances are those of the single operators (layer_refs.py)."""
import pytest
import layer_refs as R
from gpu_util import TOL_BF16, TOL_F32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
NORM_OPS = 2 * 56 + 10  # counted in test_gpu_norm.py


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


def normal(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, dt=F32, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt).cuda()


def gate_ops(z):
    return 2 * (8 + 2 * float(z.abs().max()))


def check_norm(name, y, x, w, rms=True, z=None):
    want, _, _, mag = R.norm(x, w, None, rms, EPS, z)
    R.check(name, y, want, mag, NORM_OPS + (0 if z is None else gate_ops(z)))


def check_conv(name, ys, x, w, b, init=None):
    v, y, final, mag = R.conv(x, w, b, True, init)
    # v's error and the activation's own, as counted in test_gpu_conv.py
    total = 1.1 * (w.shape[1] + 1) * mag + y.abs() * (8 + 2 * v.abs())
    R.check(name, torch.cat(ys, -1), y, total, 1.0)
    return final


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_block_with_heads(ssd, dtype):
    """norm(x + stream) -> projection -> convolution into x, B, C -> state-space
    layer -> gated norm, over a prompt and then token by token."""
    Bt, L, L0, hid, H, P, N, W = 2, 70, 64, 192, 4, 64, 64, 4
    inner, K = H * P, H * P + 2 * N
    split = (inner, N, N)
    r = normal(3)
    x, stream = r(Bt, L, hid, dt=dtype), r(Bt, L, hid)
    nw, gw, cw, cb = r(hid), r(inner), r(K, W, sc=0.5), r(K, sc=0.1)
    A, D, bias = -torch.exp(r(H)), r(H), r(H, off=-2.0)
    proj = r(hid, inner + K + H, sc=hid ** -0.5)
    n, total = ssd.norm_forward(x, nw, residual=stream, rms=True)
    R.check("sum", total, x.double().cpu() + stream.double().cpu(),
            x.double().cpu().abs() + stream.double().cpu().abs(), 1)
    check_norm("norm", n, total, nw)
    p = (n.float() @ proj).to(dtype)
    z, xbc, dt = p[..., :inner], p[..., inner:inner + K], p[..., inner + K:].contiguous()

    def scan(xs, B, C, dt):
        return ssd.forward(xs.view(Bt, -1, H, P), dt, A, B.unsqueeze(2), C.unsqueeze(2), D, chunk=64,
                           return_final_state=True, dt_bias=bias, dt_softplus=True)

    (xs, B, C), conv_state = ssd.conv_forward(xbc, cw, cb, split=split, return_final_state=True)
    final = check_conv("conv", (xs, B, C), xbc, cw, cb)
    assert torch.equal(conv_state.double().cpu(), final)
    y, state = scan(xs, B, C, dt)
    wide = lambda t: t.repeat_interleave(P, -1)  # noqa: E731
    want = R.selective(xs, wide(dt), wide(A)[:, None].expand(-1, N), B.unsqueeze(2), C.unsqueeze(2),
                       wide(D), None, None, wide(bias), True)
    assert rel(y.flatten(2), want["y"]) < (TOL_BF16 if dtype == BF else TOL_F32)
    out = ssd.norm_forward(y.flatten(2), gw, z=z, rms=True)
    check_norm("gated norm", out, y.flatten(2), gw, z=z)

    # the same, the last tokens one at a time from the states that the prompt left
    (xs0, B0, C0), cs = ssd.conv_forward(xbc[:, :L0], cw, cb, split=split, return_final_state=True)
    _, st = scan(xs0, B0, C0, dt[:, :L0].contiguous())
    for t in range(L0, L):
        nt, tt = ssd.norm_forward(x[:, t].contiguous(), nw, residual=stream[:, t].contiguous(), rms=True)
        assert torch.equal(nt, n[:, t]) and torch.equal(tt, total[:, t])
        xt, Bv, Cv = ssd.conv_step(cs, xbc[:, t], cw, cb, split=split)
        assert torch.equal(xt, xs[:, t]) and torch.equal(Bv, B[:, t]) and torch.equal(Cv, C[:, t])
        yt = ssd.step(st, xt.view(Bt, H, P), dt[:, t].contiguous(), A, Bv.unsqueeze(1), Cv.unsqueeze(1), D,
                      dt_bias=bias, dt_softplus=True)
        assert rel(yt.flatten(1), want["y"][:, t]) < (TOL_BF16 if dtype == BF else TOL_F32)
        ot = ssd.norm_forward(yt.flatten(1), gw, z=z[:, t], rms=True)
        check_norm("gated norm, token", ot, yt.flatten(1), gw, z=z[:, t])
    assert torch.equal(cs, conv_state)
    assert rel(st, state) < (TOL_BF16 if dtype == BF else TOL_F32)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_block_with_channels(ssd, dtype):
    """layer norm -> projection -> convolution -> projection -> selective scan
    with its gate: forward, every gradient, and the tokens after the prompt."""
    Bt, L, L0, hid, E, N, W, low = 2, 50, 45, 96, 192, 16, 4, 8
    r = normal(4)
    x, nw, nb = r(Bt, L, hid, dt=dtype), r(hid), r(hid)
    cw, cb = r(E, W, sc=0.5), r(E, sc=0.1)
    A, D, bias = -torch.exp(r(E, N, sc=0.5)), r(E), r(E, off=-3.0)
    w_in, w_x, w_dt = r(hid, 2 * E, sc=hid ** -0.5), r(E, low + 2 * N, sc=E ** -0.5), r(low, E, sc=low ** -0.5)
    n, mean, rstd = ssd.norm_forward(x, nw, nb, return_stats=True)
    want, _, _, mag = R.norm(x, nw, nb, False, EPS)
    R.check("norm", n, want, mag, NORM_OPS)
    p = (n.float() @ w_in).to(dtype)
    xin, z = p[..., :E], p[..., E:]
    u, conv_state = ssd.conv_forward(xin, cw, cb, return_final_state=True)
    check_conv("conv", (u,), xin, cw, cb)
    q = (u.float() @ w_x).to(dtype)
    dt = (q[..., :low].float() @ w_dt).to(dtype)
    B, C = q[..., low:low + N].unsqueeze(2), q[..., low + N:].unsqueeze(2)
    scan = dict(A=A, D=D, dt_bias=bias, dt_softplus=True)
    y, state = ssd.selective_forward(u, dt, B=B, C=C, z=z, return_final_state=True, **scan)
    dy, dstate = r(Bt, L, E, dt=dtype), r(Bt, E, N)
    want = R.selective(u, dt, A, B, C, D, z, None, bias, True, None, (dy, dstate))
    R.check("scan", y, want["y"], want["y_err"], 1)
    R.check("state", state, want["final"], want["final_err"], 1)

    # backward in the reverse order, each operator from the gradient the one before gives
    g = ssd.selective_backward(u, dt, B=B, C=C, z=z, dy=dy, dfinal_state=dstate, **scan)
    for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"):
        R.check(("scan", k), g[k], want[k], want[k + "_err"], 1)
    dq = torch.cat([g["ddt"].float() @ w_dt.t(), g["dB"].flatten(2).float(), g["dC"].flatten(2).float()], -1)
    du = (g["dx"].float() + dq @ w_x.t()).to(dtype)
    gc = ssd.conv_backward(xin, cw, cb, du)
    want, mag = R.conv_grads(xin, cw, cb, True, du)
    ops = W + 14 + (W + 1) * float(R.conv(xin, cw, cb, True)[3].max())  # counted in test_gpu_conv.py
    for k in ("dx", "dweight", "dbias"):
        R.check(("conv", k), gc[k], want[k], mag[k], ops + (Bt * L if k != "dx" else 0))
    dn = (torch.cat([gc["dx"], g["dz"]], -1).float() @ w_in.t()).to(dtype)
    gn = ssd.norm_backward(dn, x, nw, mean, rstd)
    want, mag = R.norm_grads(dn, x, nw, False, EPS)
    for k in ("dx", "dweight", "dbias"):
        R.check(("norm", k), gn[k], want[k], mag[k], 2 * NORM_OPS + (Bt * L if k != "dx" else 0))

    # the last tokens one at a time
    _, cs = ssd.conv_forward(xin[:, :L0], cw, cb, return_final_state=True)
    _, st = ssd.selective_forward(u[:, :L0], dt[:, :L0], B=B[:, :L0], C=C[:, :L0], z=z[:, :L0],
                                  return_final_state=True, **scan)
    for t in range(L0, L):
        ut = ssd.conv_step(cs, xin[:, t], cw, cb)
        assert torch.equal(ut, u[:, t])
        before = st.clone()
        yt = ssd.selective_step(st, ut, dt[:, t], B=B[:, t], C=C[:, t], z=z[:, t], **scan)
        one = R.selective(ut.unsqueeze(1), dt[:, t:t + 1], A, B[:, t:t + 1], C[:, t:t + 1], D, z[:, t:t + 1],
                          before, bias, True)
        R.check("token", yt.unsqueeze(1), one["y"], one["y_err"], 1)
        R.check("token's state", st, one["final"], one["final_err"], 1)
    assert torch.equal(cs, conv_state)


def _calls(ssd, seed):
    """One call of each operator, forward and backward, on tensors of its own."""
    r = normal(seed)
    Bt, L, E, N, W = 2, 300, 200, 16, 4
    x, dy, z = r(Bt, L, E, dt=BF), r(Bt, L, E, dt=BF), r(Bt, L, E, dt=BF)
    w, b, cw = r(E), r(E), r(E, W)
    dt, B, C = r(Bt, L, E, dt=BF, sc=0.3, off=-3.0), r(Bt, L, 1, N, dt=BF), r(Bt, L, 1, N, dt=BF)
    A, st, cs = -torch.exp(r(E, N, sc=0.5)), r(Bt, E, N), r(Bt, W - 1, E, dt=BF)
    tensors = (x, dy, z, dt, B, C, st, cs)

    def run():
        state, conv_state = st.clone(), cs.clone()
        out = [*ssd.conv_forward(x, cw, b, return_final_state=True)]
        out += ssd.conv_backward(x, cw, b, dy).values()
        out += [ssd.conv_step(conv_state, x[:, 0], cw, b), conv_state]
        out += ssd.selective_forward(x, dt, A, B, C, w, z, st, True, dt_softplus=True)
        out += ssd.selective_backward(x, dt, A, B, C, w, dy, z, st, dt_softplus=True).values()
        out += [ssd.selective_step(state, x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], w, z[:, 0]), state]
        y, mean, rstd = ssd.norm_forward(x, w, b, z=z, return_stats=True)
        out += [y, *ssd.norm_backward(dy, x, w, mean, rstd, z=z).values()]
        return [t for t in out if t is not None]
    return tensors, run


def test_other_streams(ssd):
    """Calls on two streams at once, behind work that is still going on when they
    are made: each waits for its own stream's work and disturbs no other's."""
    (ta, run_a), (tb, run_b) = _calls(ssd, 5), _calls(ssd, 6)
    want_a, want_b = run_a(), run_b()
    held = [[t.clone() for t in ts] for ts in (ta, tb)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        for ts in (ta, tb):
            for t in ts:
                t.zero_()
        torch.cuda.synchronize()
        got = [None, None]
        for i, (ts, run) in enumerate(((ta, run_a), (tb, run_b))):
            with torch.cuda.stream(streams[i]):
                for _ in range(4):
                    busy @ busy
                for t, h in zip(ts, held[i]):
                    t.copy_(h)  # the inputs only now
        for i, run in enumerate((run_a, run_b)):
            with torch.cuda.stream(streams[i]):
                got[i] = run()
        for s in streams:
            s.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got[0], want_a))
        assert all(torch.equal(g, w) for g, w in zip(got[1], want_b))


def test_two_graphs(ssd):
    """Two captured runs that share torch's graph memory, replayed in turn with
    eager calls between them."""
    (ta, run_a), (tb, run_b) = _calls(ssd, 7), _calls(ssd, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_a(), run_b()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    pool = torch.cuda.graph_pool_handle()
    for run in (run_a, run_b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(run())
        graphs.append(graph)
    for k in range(4):
        for ts in (ta, tb):
            ts[0].mul_(-0.5)
        for i, run in ((0, run_a), (1, run_b), (0, run_a))[k % 2:]:
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(g, w) for g, w in zip(outs[i], run())), (k, i)


def test_callers_workspace(ssd):
    """The stated size is enough, nothing past it is touched, and a workspace can
    serve one call after the other."""
    r = normal(9)
    Bt, L, E, N = 2, 517, 70, 16
    x, dy, B, C = r(Bt, L, E, dt=BF), r(Bt, L, E, dt=BF), r(Bt, L, 1, N, dt=BF), r(Bt, L, 1, N, dt=BF)
    dt, A, w, cw = r(Bt, L, E, dt=BF, off=-3.0), -torch.exp(r(E, N)), r(E), r(E, 4)
    from structured_state_space_ssd_amd._native import lib
    _, mean, rstd = ssd.norm_forward(x, w, return_stats=True)
    calls = [
        (lib.ssd_selective_forward_workspace_size(Bt, L, E, 1, N, 1),
         lambda ws: ssd.selective_forward(x, dt, A, B, C, w, dt_softplus=True, workspace=ws)),
        (lib.ssd_selective_backward_workspace_size(Bt, L, E, 1, N, 1),
         lambda ws: ssd.selective_backward(x, dt, A, B, C, w, dy, dt_softplus=True, workspace=ws)),
        (lib.ssd_conv_backward_workspace_size(Bt, L, E, 4, 1), lambda ws: ssd.conv_backward(x, cw, w, dy, workspace=ws)),
        (lib.ssd_norm_backward_workspace_size(Bt * L, E, 1, 1),
         lambda ws: ssd.norm_backward(dy, x, w, mean, rstd, workspace=ws))]
    most = max(need for need, _ in calls)
    for fill in (0xff, 0x7f):  # NaN, and huge values, where a call might read what it did not write
        for need, run in calls:
            buf = torch.full((most + 4096,), fill, dtype=torch.uint8, device="cuda")
            got, want = run(buf[:need]), run(None)
            assert bool((buf[need:] == fill).all())
            if isinstance(got, dict):
                assert all(want[k] is None or torch.equal(got[k], want[k]) for k in want)
            else:
                assert torch.equal(got, want)
            with pytest.raises(RuntimeError):
                run(buf[:need - 1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_far_apart(ssd, dtype):
    """Tokens and sequences whose offsets pass 2^32 elements: rows far apart in
    one allocation that only they are written to."""
    Bt, L, E, N, W = 2, 300, 24, 4, 4
    row = (1 << 24) - 8              # elements between tokens
    batch = (1 << 31) + 8            # and between sequences, whose rows interleave
    need = batch + (L - 1) * row + E
    far = torch.empty(need, dtype=dtype, device="cuda")
    r = normal(10)

    def place(near):
        view = far.as_strided((Bt, L, E), (batch, row, 1))
        view.copy_(near)
        return view
    assert (L - 1) * row > 1 << 32
    x, dy = r(Bt, L, E, dt=dtype), r(Bt, L, E, dt=dtype)
    dt, B, C = r(Bt, L, E, dt=dtype, off=-3.0), r(Bt, L, 1, N, dt=dtype), r(Bt, L, 1, N, dt=dtype)
    A, w, cw = -torch.exp(r(E, N)), r(E), r(E, W)
    xf = place(x)
    same = lambda a, b: all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)  # noqa: E731
    assert torch.equal(ssd.conv_forward(xf, cw, w), ssd.conv_forward(x, cw, w))
    assert same(ssd.conv_backward(xf, cw, w, dy), ssd.conv_backward(x, cw, w, dy))
    args = (dt, A, B, C, w)
    assert torch.equal(ssd.selective_forward(xf, *args, dt_softplus=True), ssd.selective_forward(x, *args, dt_softplus=True))
    assert same(ssd.selective_backward(xf, *args, dy, dt_softplus=True), ssd.selective_backward(x, *args, dy, dt_softplus=True))
    # the gate, the step sizes and one sequence's rows of the norm as well
    near = ssd.selective_backward(x, *args, dy, z=x, dt_softplus=True)
    assert same(ssd.selective_backward(x, *args, dy, z=xf, dt_softplus=True), near)
    assert torch.equal(ssd.norm_forward(xf[1], w, z=xf[1]), ssd.norm_forward(x[1], w, z=x[1]))
    _, mean, rstd = ssd.norm_forward(x[1], w, return_stats=True)
    assert same(ssd.norm_backward(dy[1], xf[1], w, mean, rstd), ssd.norm_backward(dy[1], x[1], w, mean, rstd))


def test_conv_packed_padding(ssd):
    """Rows behind the last sequence change nothing in front of them, whatever
    they hold, nor in the states."""
    r = normal(11)
    L, K, W, cu = 90, 40, 4, [0, 3, 3, 50, 70]
    w, b = r(K, W), r(K)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    x = r(1, L, K, dt=BF)
    want, final = ssd.conv_forward(x[:, :cu[-1]], w, b, cu_seqlens=c, return_final_state=True)
    for fill in (0.0, float("nan"), float("inf")):
        x[:, cu[-1]:] = fill
        y, f = ssd.conv_forward(x, w, b, cu_seqlens=c, return_final_state=True)
        assert torch.equal(y[:, :cu[-1]], want) and torch.equal(f, final)
