"""The recurrence, the block norm and dropout run together with the convolution, as a
recurrent model runs them: a prompt, the tokens after it and a training step; on other
streams, in graphs, with a caller's workspaces and with offsets past 2^32. Each operator is
checked against its plain 64-bit form on the inputs that it got."""
import pytest
import block_refs as B
import layer_refs as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
OPS = 122  # a norm (test_gpu_norm.py)


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


def normal(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, dt=F32, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt).cuda()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_recurrent_blocks(ssd, dtype):
    """Two blocks of projection -> convolution -> recurrence -> projection -> block norm with
    dropout over a prompt, their gradients, then the last tokens one at a time without it."""
    Bt, L, L0, hid, E, W, p = 2, 70, 64, 96, 130, 4, 0.2
    r = normal(5)
    stream, x = r(Bt, L, hid), r(Bt, L, hid, dt=dtype)
    blocks = [dict(cw=r(E, W, sc=0.5), cb=r(E, sc=0.1), decay=r(E, off=-4.0), win=r(hid, 4 * E, sc=hid ** -0.5),
                   wout=r(E, hid, sc=E ** -0.5), pw=r(hid, off=1.0, sc=0.2), nw=r(hid, off=1.0, sc=0.2), sc=r(hid, sc=0.3))
              for _ in range(2)]

    def mixer(b, h):
        q = (h.float() @ b["win"]).to(dtype)  # x, both gates' inputs and the output gate
        u = ssd.conv_forward(q[..., :E], b["cw"], b["cb"])
        rec = dict(x=u, r=q[..., E:2 * E], i=q[..., 2 * E:3 * E], decay=b["decay"], z=q[..., 3 * E:])
        y, final, states = ssd.recurrence_forward(**rec, return_final_state=True, return_states=True)
        return q, rec, y, final, states

    h, s, kept = x, stream, []
    for n, b in enumerate(blocks):
        q, rec, y, final, states = mixer(b, h)
        want = B.recurrence(**rec)
        R.check((n, "scan"), y, want["y"], want["y_err"], 1)
        o = (y.float() @ b["wout"]).to(dtype)
        kw = dict(weight=b["nw"], post_weight=b["pw"], scale=b["sc"], p=p, rng=(9, n), branch_scale=0.5)
        h2, s2, stats = ssd.block_norm_forward(o, s, **kw, rms=True, return_stats=True)
        ref = B.Block(o, s, weight=b["nw"], post_weight=b["pw"], scale=b["sc"], p=p, rng=(9, n), beta=0.5, rms=True)
        R.check((n, "sum"), s2, ref.total, ref.total_mag, OPS + 6)
        R.check((n, "norm"), h2, *ref.y(s2), OPS)
        kept.append((h, s, q, rec, states, o, kw, s2, stats, ref))
        h, s = h2, s2

    dh, ds = r(Bt, L, hid, dt=dtype), r(Bt, L, hid)
    for n in (1, 0):
        b = blocks[n]
        h, s, q, rec, states, o, kw, s2, stats, ref = kept[n]
        g = ssd.block_norm_backward(dh, ds, o, s2, stats, **kw)
        want, mag = ref.grads(dh, ds, s2)
        for k in want:
            R.check((n, k), g[k], want[k], mag[k], 4 * OPS + 16 + (Bt * L if k not in ("dx", "dresidual") else 0))
        dy = (g["dx"].float() @ b["wout"].t()).to(dtype)
        gr = ssd.recurrence_backward(**rec, dy=dy, states=states)
        want = B.recurrence(**rec, grads=(dy, None))
        for k in ("dx", "dr", "di", "dz", "ddecay"):
            R.check((n, k), gr[k], want[k], want[k + "_err"], 1)
        gc = ssd.conv_backward(q[..., :E], b["cw"], b["cb"], gr["dx"])
        dq = torch.cat([gc["dx"], gr["dr"], gr["di"], gr["dz"]], -1)
        dh, ds = (dq.float() @ b["win"].t()).to(dtype), g["dresidual"]

    # the last tokens one at a time, in a block without dropout
    b = blocks[0]
    q, rec, y, _, _ = mixer(b, x)
    _, cs = ssd.conv_forward(q[:, :L0, :E], b["cw"], b["cb"], return_final_state=True)
    _, st = ssd.recurrence_forward(**{k: v if v.dim() == 1 else v[:, :L0] for k, v in rec.items()}, return_final_state=True)
    for t in range(L0, L):
        u = ssd.conv_step(cs, q[:, t, :E], b["cw"], b["cb"])
        assert torch.equal(u, rec["x"][:, t])
        before = st.clone()
        yt = ssd.recurrence_step(st, **{k: v if v.dim() == 1 else v[:, t] for k, v in rec.items()})
        one = B.recurrence(**{k: v if v.dim() == 1 else v[:, t:t + 1] for k, v in rec.items()}, init=before)
        R.check("token", yt, one["y"][:, 0], one["y_err"][:, 0], 1)
        R.check("token's state", st, one["final"], one["final_err"], 1)
        o = (yt.float() @ b["wout"]).to(dtype)
        ht, stt = ssd.block_norm_forward(o, stream[:, t].contiguous(), b["nw"], post_weight=b["pw"], scale=b["sc"], rms=True)
        ref = B.Block(o, stream[:, t], weight=b["nw"], post_weight=b["pw"], scale=b["sc"], rms=True)
        R.check("token's sum", stt, ref.total, ref.total_mag, OPS + 6)
        R.check("token's norm", ht, *ref.y(stt), OPS)


def _calls(ssd, seed):
    """One call of each operator, forward and backward, on tensors of its own."""
    r = normal(seed)
    Bt, L, E = 2, 1300, 200
    a = dict(x=r(Bt, L, E, dt=BF), r=r(Bt, L, E, dt=BF), i=r(Bt, L, E, dt=BF), decay=r(E, off=-3.0), z=r(Bt, L, E, dt=BF))
    dy, st, w, k = r(Bt, L, E, dt=BF), r(Bt, E), r(E, off=1.0), r(E)
    cu = torch.tensor([0, 100, 100, 777, L], dtype=torch.int32, device="cuda")
    rng = torch.tensor([seed, 3], device="cuda")
    tensors = (a["x"], a["r"], a["i"], a["z"], dy, st)

    def run():
        state = st.clone()
        one = {n: v if v.dim() == 1 else v[:, 0] for n, v in a.items()}
        packed = {n: v if v.dim() == 1 else v[:1] for n, v in a.items()}
        y, final, states = ssd.recurrence_forward(**a, init_state=st, return_final_state=True, return_states=True)
        out = [y, final, *ssd.recurrence_backward(**a, dy=dy, init_state=st, states=states).values()]
        out += ssd.recurrence_backward(**a, dy=dy, dfinal_state=st).values()
        out += ssd.recurrence_forward(**packed, cu_seqlens=cu, return_final_state=True)
        out += ssd.recurrence_backward(**packed, dy=dy[:1], cu_seqlens=cu).values()
        out += [ssd.recurrence_step(state, **one), state, ssd.dropout(dy, 0.3, rng)]
        kw = dict(weight=w, post_weight=k, post_bias=w, scale=w, z=a["z"], p=0.1, rng=rng)
        h, s, stats = ssd.block_norm_forward(a["x"], dy, **kw, return_stats=True)
        out += [h, s, *ssd.block_norm_backward(dy, s, a["x"], s, stats, **kw).values()]
        return [t for t in out if t is not None]
    return tensors, run


def test_other_streams(ssd):
    """Calls on two streams at once, behind work that is still going on when they are
    made: each waits for its own stream's work and disturbs no other's."""
    (ta, run_a), (tb, run_b) = _calls(ssd, 5), _calls(ssd, 6)
    want = [run_a(), run_b()]
    held = [[t.clone() for t in ts] for ts in (ta, tb)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        for t in (*ta, *tb):
            t.zero_()
        torch.cuda.synchronize()
        got = [None, None]
        for i, ts in enumerate((ta, tb)):
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
        for i in range(2):
            assert all(torch.equal(g, w) for g, w in zip(got[i], want[i]))


def test_two_graphs(ssd):
    """Two captured runs that share torch's graph memory, replayed in turn with eager calls
    between them."""
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
    """The stated size is enough, nothing past it is touched, and a workspace can serve one
    call after the other, whatever it holds."""
    r = normal(9)
    from structured_state_space_ssd_amd._native import lib
    Bt, L, E = 1, 4099, 70
    a = dict(x=r(Bt, L, E, dt=BF), r=r(Bt, L, E, dt=BF), i=r(Bt, L, E, dt=BF), decay=r(E, off=-3.0))
    dy, w = r(Bt, L, E, dt=BF), r(E)
    cu = torch.tensor([0, 64, 65, 3000, L], dtype=torch.int32, device="cuda")
    _, states = ssd.recurrence_forward(**a, return_states=True)
    _, total, stats = ssd.block_norm_forward(a["x"], dy, w, return_stats=True)
    calls = [
        (lib.ssd_recurrence_forward_workspace_size(Bt, L, E, 0, 1), lambda ws: ssd.recurrence_forward(**a, workspace=ws)),
        (lib.ssd_recurrence_forward_workspace_size(Bt, L, E, 1, 1),
         lambda ws: ssd.recurrence_forward(**a, cu_seqlens=cu, workspace=ws)),
        (lib.ssd_recurrence_backward_workspace_size(Bt, L, E, 0, 1, 1),
         lambda ws: ssd.recurrence_backward(**a, dy=dy, states=states, workspace=ws)),
        (lib.ssd_recurrence_backward_workspace_size(Bt, L, E, 1, 0, 1),
         lambda ws: ssd.recurrence_backward(**a, dy=dy, cu_seqlens=cu, workspace=ws)),
        (lib.ssd_block_norm_backward_workspace_size(L, E, 1),
         lambda ws: ssd.block_norm_backward(dy, None, a["x"], total, stats, w, workspace=ws))]
    most = max(need for need, _ in calls)
    for fill in (0xff, 0x7f):  # NaN, and huge values, where a call might read what it did not write
        for need, run in calls:
            assert need > 0
            buf = torch.full((most + 4096,), fill, dtype=torch.uint8, device="cuda")
            got, want = run(buf[:need]), run(None)
            assert bool((buf[need:] == fill).all())
            if isinstance(got, dict):
                assert all(want[k] is None or torch.equal(got[k], want[k]) for k in want)
            else:
                assert torch.equal(got, want)
    for need, run in calls[:4]:
        with pytest.raises(RuntimeError):
            run(buf[:need - 1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_far_apart(ssd, dtype):
    """Tokens and sequences whose offsets pass 2^32 elements."""
    Bt, L, E = 2, 300, 40
    row, batch = (1 << 24) - 8, (1 << 31) + 8  # the sequences' rows interleave
    far = torch.empty(batch + (L - 1) * row + E, dtype=dtype, device="cuda")
    r = normal(10)
    near = [r(Bt, L, E, dt=dtype) for _ in range(4)]
    decay, dy, st = r(E, off=-3.0), r(Bt, L, E, dt=dtype), r(Bt, E)
    names = ("x", "r", "i", "z")
    a = dict(zip(names, near), decay=decay)
    y, g = ssd.recurrence_forward(**a), ssd.recurrence_backward(**a, dy=dy)
    for k in names:
        view = far.as_strided((Bt, L, E), (batch, row, 1))
        view.copy_(a[k])
        b = {**a, k: view}
        assert torch.equal(ssd.recurrence_forward(**b), y)
        h = ssd.recurrence_backward(**b, dy=dy)
        assert all(torch.equal(g[n], h[n]) for n in g if g[n] is not None), k
        s1, s2 = st.clone(), st.clone()
        one = lambda d: {n: v if v.dim() == 1 else v[:, -1] for n, v in d.items()}  # noqa: E731
        assert torch.equal(ssd.recurrence_step(s1, **one(a)), ssd.recurrence_step(s2, **one(b))) and torch.equal(s1, s2)
