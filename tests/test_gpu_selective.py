"""The selective scan on the GPU against its plain 64-bit form, whose bounds
follow the roundings through the recurrence (layer_refs.selective)."""
import pytest
import layer_refs as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


def make(Bt, L, E, N, G, dtype, seed, D=True, z=True, init=True, sliced=0, soft=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=dtype, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt).cuda()  # noqa: E731
    bc = r(Bt, L, sliced + 2 * G * N, sc=N ** -0.5)
    a = dict(x=r(Bt, L, E + sliced)[..., sliced:],
             dt=r(Bt, L, E, sc=0.5) if soft else (torch.rand(Bt, L, E, generator=g) * 0.1).to(dtype).cuda(),
             A=-torch.exp(torch.rand(E, N, generator=g) * 2.77).cuda(),
             B=bc[..., sliced:sliced + G * N].unflatten(-1, (G, N)),
             C=bc[..., sliced + G * N:].unflatten(-1, (G, N)))
    a["D"] = r(E, dt=F32) if D else None
    a["z"] = r(Bt, L, 2 * E)[..., E:] if z else None
    a["init_state"] = r(Bt, E, N, dt=F32) if init else None
    a["dt_bias"] = r(E, dt=F32, off=-3.0) if soft else None
    a["dt_softplus"] = soft
    return a, r


def ref(a, **kw):
    return R.selective(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["init_state"],
                       a["dt_bias"], a["dt_softplus"], a.get("dt_limit"), **kw)


def check(name, got, want, key):
    R.check((name, key), got, want[key], want[key + "_err"], 1.0)


# (batch, tokens, channels, state, groups): one token, tiles of 8 to 32 tokens and one
# more or less, states below, at and past each of the kernels' sizes, channels that
# leave a workgroup part empty, groups whose channels end inside one
SIZES = [(1, 1, 1, 1, 1), (2, 1, 64, 16, 1), (1, 2, 5, 3, 1), (2, 7, 256, 4, 1), (1, 9, 300, 2, 1),
         (1, 15, 130, 8, 2), (2, 17, 128, 7, 1), (1, 31, 64, 16, 1), (2, 33, 70, 16, 2),
         (1, 32, 96, 13, 3), (1, 33, 40, 32, 1), (2, 65, 66, 24, 2), (1, 40, 20, 64, 1),
         (1, 67, 34, 50, 2), (3, 100, 12, 16, 4)]
# few channels over many tokens: cut into segments (the last one shorter than the others)
# (260, 270: a few more workgroups than CUs, of which only those few are cut)
LONG = [(1, 300, 64, 16, 1), (1, 1000, 8, 16, 1), (2, 517, 33, 5, 1), (1, 700, 16, 64, 1), (1, 260, 300, 3, 2)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES + LONG + [(260, 130, 8, 16, 1), (270, 41, 6, 3, 2)], ids=str)
def test_selective_forward(ssd, size, dtype):
    for D, z, init, sliced, soft in ((True, True, True, 5, True), (False, False, False, 0, False),
                                     (True, False, True, 8, False)):
        a, _ = make(*size, dtype, sum(size), D, z, init, sliced, soft)
        want = ref(a)
        y, final = ssd.selective_forward(**a, return_final_state=True)
        check(size, y, want, "y")
        check(size, final, want, "final")
        assert torch.equal(ssd.selective_forward(**a), y)


def test_selective_clamp(ssd):
    a, _ = make(2, 50, 40, 16, 1, F32, 1)
    a["dt_limit"] = (0.02, 0.08)
    want = ref(a)
    y, final = ssd.selective_forward(**a, return_final_state=True)
    check("clamp", y, want, "y")
    check("clamp", final, want, "final")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [(5, 3, 7, 1, 1), (2, 4, 70, 16, 2), (3, 2, 64, 6, 1), (1, 5, 33, 64, 1), (2, 3, 20, 21, 4)], ids=str)
def test_selective_step(ssd, size, dtype):
    """Token by token from the initial state: every token's y and the last state."""
    for D, z, sliced, soft in ((True, True, 5, True), (False, False, 0, False)):
        a, _ = make(*size, dtype, sum(size), D, z, True, sliced, soft)
        want = ref(a)
        state = a.pop("init_state").clone()
        for t in range(size[1]):
            cut = {k: (v[:, t] if k in ("x", "dt", "B", "C", "z") and v is not None else v) for k, v in a.items()}
            y = ssd.selective_step(state, **cut)
            R.check((size, t), y, want["y"][:, t], want["y_err"][:, t], 1.0)
        check(size, state, want, "final")


def test_selective_goes_on(ssd):
    """A prompt in two parts, then single tokens, against the whole at once."""
    a, _ = make(2, 200, 72, 16, 1, F32, 9)
    want = ref(a)
    cut = lambda s: {k: (v[:, s] if k in ("x", "dt", "B", "C", "z") else v) for k, v in a.items()}  # noqa: E731
    y0, st = ssd.selective_forward(**cut(slice(0, 77)), return_final_state=True)
    second = dict(cut(slice(77, 190)), init_state=st)
    y1, st = ssd.selective_forward(**second, return_final_state=True)
    ys = [y0, y1]
    for t in range(190, 200):
        one = cut(t)
        one.pop("init_state")
        ys.append(ssd.selective_step(st, **one)[:, None])
    check("parts", torch.cat(ys, 1), want, "y")
    check("parts", st, want, "final")


def test_selective_strong_and_no_decay(ssd):
    """Decays that underflow to zero, and none at all (A = 0, growing states)."""
    a, _ = make(1, 120, 64, 16, 1, F32, 4, soft=False)
    a["A"] = a["A"] * 1e4
    want = ref(a)
    check("strong", ssd.selective_forward(**a), want, "y")
    a["A"] = torch.zeros_like(a["A"])
    want = ref(a)
    check("none", ssd.selective_forward(**a), want, "y")


@pytest.mark.parametrize("size", [(2, 33, 70, 16, 1), (1, 700, 16, 13, 1)], ids=str)
def test_selective_no_memory(ssd, size):
    """A = -inf forgets everything at a step and nothing where the step size is zero
    (the rows past a tile's end among them); -1e30 is the same to any step size here."""
    a, r = make(*size, F32, 5, soft=False)
    a["dt"] = a["dt"].clamp(min=1e-3)
    dy = r(*size[:3])
    a["A"][:, ::2] = -1e30
    y, final = ssd.selective_forward(**a, return_final_state=True)
    check("finite", y, ref(a), "y")
    grads = ssd.selective_backward(**a, dy=dy)
    b = dict(a, A=a["A"].clone())
    b["A"][:, ::2] = -float("inf")
    y2, final2 = ssd.selective_forward(**b, return_final_state=True)
    assert torch.equal(y, y2) and torch.equal(final, final2)
    got = ssd.selective_backward(**b, dy=dy)
    assert all(torch.equal(got[k], grads[k]) for k in grads if grads[k] is not None)
    state = a["init_state"].clone()
    one = {k: (v[:, 0] if k in ("x", "dt", "B", "C", "z") and v is not None else v) for k, v in b.items()
           if k != "init_state"}
    ssd.selective_step(state, **dict(one, dt=torch.zeros_like(one["dt"])))
    assert torch.equal(state, a["init_state"])


def test_selective_nan_stays_in_its_channel(ssd):
    a, _ = make(1, 300, 64, 16, 1, F32, 4)
    a["x"] = a["x"].clone()
    a["x"][0, 100, 7] = float("nan")
    y, final = ssd.selective_forward(**a, return_final_state=True)
    assert y[0, 100:, 7].isnan().all() and final[0, 7].isnan().all()
    y[0, 100:, 7] = 0
    final[0, 7] = 0
    assert y.isfinite().all() and final.isfinite().all()


GRADS = ("dx", "ddt", "dz", "dB", "dC", "dA", "dD", "dinit", "ddt_bias")


def check_grads(name, got, want):
    for k in GRADS:
        if got.get(k) is not None:
            check(name, got[k], want, k)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES + LONG, ids=str)
def test_selective_backward(ssd, size, dtype):
    for D, z, init, sliced, soft in ((True, True, True, 5, True), (False, False, False, 0, False),
                                     (True, False, True, 8, True)):
        a, r = make(*size, dtype, sum(size), D, z, init, sliced, soft)
        dy = r(*size[:3])
        dfinal = r(size[0], size[2], size[3], dt=F32) if init else None
        want = ref(a, grads=(dy, dfinal))
        got = ssd.selective_backward(**a, dy=dy, dfinal_state=dfinal)
        assert ("dz" in got) == z and ("ddt_bias" in got) == soft
        check_grads((size, z), got, want)
        again = ssd.selective_backward(**a, dy=dy, dfinal_state=dfinal, want_dinit=False)
        assert again["dinit"] is None
        assert all(torch.equal(got[k], again[k]) for k in got if k != "dinit")


def test_selective_backward_clamp(ssd):
    a, r = make(2, 50, 40, 16, 1, F32, 1)
    a["dt_limit"] = (0.02, 0.08)
    dy = r(2, 50, 40)
    want = ref(a, grads=(dy, None))
    got = ssd.selective_backward(**a, dy=dy)
    assert (got["ddt"] == 0).any()
    check_grads("clamp", got, want)


def test_selective_differences(ssd):
    """The gradient is the loss's slope: central differences of the 64-bit form."""
    a, r = make(2, 20, 9, 5, 3, F32, 11)
    dy, dfinal = r(2, 20, 9), r(2, 9, 5)
    got = ssd.selective_backward(**a, dy=dy, dfinal_state=dfinal)

    def loss(key, at, h):
        b = {k: (v.double().cpu().clone() if torch.is_tensor(v) else v) for k, v in a.items()}
        b[key][at] += h
        o = ref(b)
        return float((o["y"] * dy.double().cpu()).sum() + (o["final"] * dfinal.double().cpu()).sum())

    h = 1e-4
    for key, grad, at in (("x", "dx", (1, 7, 3)), ("dt", "ddt", (0, 19, 8)), ("dt", "ddt", (1, 0, 0)),
                          ("A", "dA", (4, 2)), ("B", "dB", (0, 11, 2, 4)), ("C", "dC", (1, 5, 0, 0)),
                          ("D", "dD", (6,)), ("z", "dz", (1, 13, 5)), ("init_state", "dinit", (0, 3, 1)),
                          ("dt_bias", "ddt_bias", (2,))):
        slope = (loss(key, at, h) - loss(key, at, -h)) / (2 * h)
        assert abs(slope - float(got[grad][at])) < 2e-4 * max(1.0, abs(slope)), (key, slope, float(got[grad][at]))


def test_selective_captured(ssd):
    a, r = make(1, 300, 70, 16, 1, BF, 2)
    dy = r(1, 300, 70)
    one = {k: (v[:, 0] if k in ("x", "dt", "B", "C", "z") else v) for k, v in a.items() if k != "init_state"}
    state = a["init_state"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssd.selective_backward(**a, dy=dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, fin = ssd.selective_forward(**a, return_final_state=True)
        g = ssd.selective_backward(**a, dy=dy)
        ys = ssd.selective_step(state, **one)
    for k in range(4):
        a["x"].copy_(torch.randn(a["x"].shape).to(BF))
        state.copy_(a["init_state"])
        graph.replay()
        torch.cuda.synchronize()
        ey, efin = ssd.selective_forward(**a, return_final_state=True)
        eg = ssd.selective_backward(**a, dy=dy)
        st = a["init_state"].clone()
        es = ssd.selective_step(st, **one)
        assert torch.equal(y, ey) and torch.equal(fin, efin) and torch.equal(ys, es) and torch.equal(state, st)
        assert all(torch.equal(g[n], eg[n]) for n in eg)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("soft", [True, False], ids=["softplus", "raw"])
@pytest.mark.parametrize("size", [(2, 40, 70, 16, 1), (1, 700, 16, 13, 1)], ids=str)
def test_selective_clamp_keeps_nan(ssd, size, soft, dtype):
    """A step size that is not a number stays one through the clamp, as without
    it: in its channel from its token on, in the gradients, and in single tokens."""
    a, r = make(*size, dtype, 6, soft=soft)
    t, e = 20, 5
    a["dt"] = a["dt"].clone()
    a["dt"][0, t, e] = float("nan")
    dy = r(*size[:3])
    free = ssd.selective_backward(**a, dy=dy)
    a["dt_limit"] = (0.02, 0.08)
    y, final = ssd.selective_forward(**a, return_final_state=True)
    bad = torch.zeros(y.shape, dtype=torch.bool)
    bad[0, t:, e] = True
    assert torch.equal(y.isnan().cpu(), bad) and final[0, e].isnan().all()
    final[0, e] = 0
    assert final.isfinite().all()
    got = ssd.selective_backward(**a, dy=dy)
    assert got["ddt"][0, t, e].isnan() and (not soft or got["ddt_bias"][e].isnan())
    for k in got:
        if k != "ddt" and got[k] is not None:  # (outside the bounds ddt is 0, whatever comes back)
            assert torch.equal(got[k].isnan(), free[k].isnan()), k
    state = a["init_state"].clone()
    one = {k: (v[:, t] if k in ("x", "dt", "B", "C", "z") else v) for k, v in a.items() if k != "init_state"}
    ys = ssd.selective_step(state, **one)
    bad = torch.zeros(ys.shape, dtype=torch.bool)
    bad[0, e] = True
    assert torch.equal(ys.isnan().cpu(), bad) and state[0, e].isnan().all()


def test_selective_step_reads_batch_strides_only(ssd):
    """Whatever the strides' token members hold: a single token has none."""
    import ctypes
    from structured_state_space_ssd_amd import _native
    Bt, E, N = 3, 20, 6
    a, _ = make(Bt, 1, E, N, 1, F32, 8, soft=False)
    one = {k: v[:, 0].contiguous() for k, v in a.items() if k in ("x", "dt", "B", "C")}
    state, again = a["init_state"].clone(), a["init_state"].clone()
    want = ssd.selective_step(state, one["x"], one["dt"], a["A"], one["B"], one["C"])
    y = torch.empty_like(want)
    for token in (-1, 1 << 40):
        st = _native.SsdSelectiveStrides(E, token, E, token, 0, token, N, token, N, token)
        again.copy_(a["init_state"])
        rc = _native.lib.ssd_selective_step(
            again.data_ptr(), one["x"].data_ptr(), one["dt"].data_ptr(), a["A"].data_ptr(), one["B"].data_ptr(),
            one["C"].data_ptr(), None, None, Bt, E, 1, N, 0, y.data_ptr(), ctypes.byref(st), None,
            _native.stream_handle())
        assert rc == 0 and torch.equal(y, want) and torch.equal(again, state)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 5000, 6, 3, 1), (2, 2100, 3, 64, 1)], ids=str)
def test_selective_many_segments(ssd, size, dtype):
    """Few channels over very many tokens: up to 125 segments, which the last one folds
    one after another (and the first one's adjoint from behind)."""
    a, r = make(*size, dtype, 12)
    dy, dfinal = r(*size[:3]), r(size[0], size[2], size[3], dt=F32)
    want = ref(a, grads=(dy, dfinal))
    y, final = ssd.selective_forward(**a, return_final_state=True)
    check(size, y, want, "y")
    check(size, final, want, "final")
    check_grads(size, ssd.selective_backward(**a, dy=dy, dfinal_state=dfinal), want)


@pytest.mark.parametrize("size", [(1100, 70, 8, 3, 1), (1030, 40, 6, 13, 2)], ids=str)
def test_selective_uncut_backward(ssd, size):
    """So many sequences that the backward walks each in one piece, over several tiles."""
    a, r = make(*size, F32, 13)
    dy, dfinal = r(*size[:3]), r(size[0], size[2], size[3])
    check_grads(size, ssd.selective_backward(**a, dy=dy, dfinal_state=dfinal), ref(a, grads=(dy, dfinal)))


def test_selective_one_token_far_apart(ssd):
    """One token of many sequences out of a tensor with the tokens in front."""
    Bt, E, N = 3, 40, 6
    a, r = make(Bt, 1, E, N, 1, F32, 9)
    dy = r(Bt, 1, E)
    y, final = ssd.selective_forward(**a, return_final_state=True)
    grads = ssd.selective_backward(**a, dy=dy)
    for k in ("x", "dt", "z", "B", "C"):
        t = a[k]
        a[k] = t.as_strided(t.shape, (t.stride(0), 1 << 30) + t.stride()[2:])
    y2, final2 = ssd.selective_forward(**a, return_final_state=True)
    again = ssd.selective_backward(**a, dy=dy)
    assert torch.equal(y, y2) and torch.equal(final, final2)
    assert all(torch.equal(grads[k], again[k]) for k in grads)
