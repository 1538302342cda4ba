"""The gated recurrence on the GPU against its plain 64-bit form, whose errors are
counted in block_refs.py."""
import pytest
import block_refs as B
import layer_refs as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


def normal(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, dt=F32, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt).cuda()


def make(Bt, L, E, dtype, gated, gate, pad=0, seed=0):
    r = normal(seed + Bt + L + E)
    a = dict(x=r(Bt, L, E + pad, dt=dtype)[..., pad:], r=r(Bt, L, E + pad, dt=dtype)[..., :E], i=None, decay=None)
    if gated:
        a["i"], a["decay"] = r(Bt, L, E, dt=dtype), r(E, sc=2.0, off=-4.0)
    else:
        a["r"] = -a["r"].abs()
    a["z"] = r(Bt, L, 2 * E, dt=dtype)[..., E:] if gate else None
    return a, r


def check_all(name, got, want, keys):
    for k in keys:
        R.check((name, k), got[k], want[k], want[k + "_err"], 1.0)


# (batch, tokens, channels): one token, parts of strands (8 tokens), wavefronts (32), tiles
# of 1 to 4 wavefronts, ragged ones, odd channels around a workgroup's 32, one tile to a unit
# and many, in one group of tiles and several, more workgroups than run at once
SIZES = [(1, 1, 1), (3, 1, 70), (2, 7, 33), (1, 8, 32), (2, 31, 31), (1, 33, 66), (5, 64, 129), (1, 130, 700),
         (2, 517, 40), (1, 2050, 34), (17, 100, 1000), (1, 4100, 3), (600, 40, 33), (8, 700, 1000)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_recurrence(ssd, size, dtype):
    Bt, L, E = size
    for gated, gate, ends, pad in ((True, True, True, 3), (True, False, False, 0), (False, False, True, 5),
                                   (False, True, False, 0)):
        if L * Bt * E > 200000 and gate != gated:
            continue
        a, r = make(Bt, L, E, dtype, gated, gate, pad)
        init = r(Bt, E) if ends else None
        dy, dfinal = r(Bt, L, E, dt=dtype), r(Bt, E) if ends else None
        want = B.recurrence(*a.values(), init, 8.0, None, (dy, dfinal))
        y, final, states = ssd.recurrence_forward(**a, init_state=init, return_final_state=True, return_states=True)
        check_all((size, gated), dict(y=y, final=final, states=states), want, ("y", "final", "states"))
        got = ssd.recurrence_backward(**a, dy=dy, init_state=init, dfinal_state=dfinal, states=states)
        keys = [k for k in got if got[k] is not None]
        assert set(keys) == {"dx", "dr"} | ({"di", "ddecay"} if gated else set()) | ({"dz"} if gate else set()) | (
            {"dinit"} if ends else set())
        check_all((size, gated), got, want, keys)
        again = ssd.recurrence_backward(**a, dy=dy, init_state=init, dfinal_state=dfinal)
        assert all(torch.equal(got[k], again[k]) for k in keys)  # with states of its own, and every time


@pytest.mark.parametrize("gated", [True, False])
def test_recurrence_long(ssd, gated):
    """Hundreds of tiles one after the other, the state entering each through many groups."""
    a, r = make(1, 30001, 40, BF, gated, False)
    if not gated:
        a["r"] = (a["r"].float() * 1e-3).bfloat16()  # a state that keeps thousands of tokens
    dy, init, dfinal = r(1, 30001, 40, dt=BF), r(1, 40), r(1, 40)
    want = B.recurrence(*a.values(), init, 8.0, None, (dy, dfinal))
    y, final, states = ssd.recurrence_forward(**a, init_state=init, return_final_state=True, return_states=True)
    check_all(gated, dict(y=y, final=final, states=states), want, ("y", "final", "states"))
    got = ssd.recurrence_backward(**a, dy=dy, init_state=init, dfinal_state=dfinal, states=states)
    check_all(gated, got, want, [k for k in got if got[k] is not None])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 2, 1], ids=["dense", "words", "off words"])
@pytest.mark.parametrize("packed", [False, True], ids=["batch", "packed"])
def test_recurrence_pairs_of_channels(ssd, packed, pad, dtype):
    """Whole tiles whose pairs of channels lie on 32-bit words, and beside them."""
    Bt, L, E, cu = (1, 520, 96, [0, 200, 520]) if packed else (3, 260, 96, None)
    a, r = make(Bt, L, E, dtype, True, True, pad)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None
    init, dy = None if packed else r(Bt, E), r(Bt, L, E, dt=dtype)
    want = B.recurrence(*a.values(), init, 8.0, cu, (dy, None))
    y, final, states = ssd.recurrence_forward(**a, init_state=init, cu_seqlens=c, return_final_state=True,
                                              return_states=True)
    check_all((packed, pad), dict(y=y, final=final), want, ("y", "final"))
    got = ssd.recurrence_backward(**a, dy=dy, init_state=init, cu_seqlens=c, states=states)
    check_all((packed, pad), got, want, [k for k in got if got[k] is not None])


CUS = [[0, 40], [0, 0, 1, 2, 2, 15, 31, 40, 40], [0, 3, 300, 300, 301, 511, 700], [0, 64, 1000, 1100],
       list(range(0, 1031, 103)), [7, 9, 64, 200, 300], [0, 2049]]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cu", CUS, ids=lambda c: str(c)[:40])
def test_recurrence_packed(ssd, cu, dtype):
    L, nseq = cu[-1], len(cu) - 1
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for gated, gate, E in ((True, True, 35), (False, False, 70), (True, False, 64)):
        a, r = make(1, L, E, dtype, gated, gate, 3)
        dy, dfinal = r(1, L, E, dt=dtype), r(nseq, E) if gate else None
        want = B.recurrence(*a.values(), None, 8.0, cu, (dy, dfinal))
        y, final, states = ssd.recurrence_forward(**a, cu_seqlens=c, return_final_state=True, return_states=True)
        check_all((cu, gated), dict(y=y, final=final), want, ("y", "final"))
        for s in (states, None):
            got = ssd.recurrence_backward(**a, dy=dy, dfinal_state=dfinal, cu_seqlens=c, states=s)
            check_all((cu, gated), got, want, [k for k in got if got[k] is not None])


def test_recurrence_packed_keeps_apart(ssd):
    """What is not a number or infinite in one sequence, or in the rows behind the last
    one, reaches no other sequence and no other's gradient; rows behind give zeros."""
    r = normal(3)
    L, E, cu = 300, 40, [0, 5, 70, 70, 133, 200]
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for dtype in (BF, F32):
        a, _ = make(1, L, E, dtype, True, True)
        dy = r(1, L, E, dt=dtype)
        clean = {k: v if v.dim() == 1 else v.clone() for k, v in a.items()}
        for bad in (float("nan"), float("inf")):
            for k in ("x", "r", "i", "z"):
                a[k][:, 200:] = bad
            a["x"][:, 10] = bad      # in the second sequence
            a["x"][:, 132] = bad     # the fourth's last token
            dyb = dy.clone()
            dyb[:, 200:] = bad
            y, final = ssd.recurrence_forward(**a, cu_seqlens=c, return_final_state=True)
            want, wfinal = ssd.recurrence_forward(**clean, cu_seqlens=c, return_final_state=True)
            g, w = ssd.recurrence_backward(**a, dy=dyb, cu_seqlens=c), ssd.recurrence_backward(**clean, dy=dy, cu_seqlens=c)
            for p, q in ((0, 5), (70, 132), (133, 200)):
                assert torch.equal(y[:, p:q], want[:, p:q])
                for k in ("dx", "dr", "di", "dz"):
                    assert torch.equal(g[k][:, p:q], w[k][:, p:q]), (k, p)
            assert bool((y[:, 200:] == 0).all()) and all(bool((g[k][:, 200:] == 0).all()) for k in ("dx", "dr", "di", "dz"))
            assert all(torch.equal(final[k], wfinal[k]) for k in (0, 2, 4)) and not bool(final[1].isfinite().any())


def test_recurrence_extreme_gates(ssd):
    """Gates and decays at their ends: open and shut gates, channels that keep everything
    and nothing; no result that the formula has finite is anything else."""
    L = 50
    decay = torch.tensor([-200.0, -100.0, -30.0, -21.0, -19.0, 0.0, 30.0, 200.0], device="cuda")
    E = len(decay)
    r = normal(4)
    x, dy = r(1, L, E), r(1, L, E)
    for rv in (0.0, -20.0, -100.0, -1e4, float("-inf"), 40.0, 1e4, float("inf")):
        for iv in (0.0, -200.0, 50.0):
            a = dict(x=x, r=torch.full_like(x, rv), i=torch.full_like(x, iv), decay=decay)
            y = ssd.recurrence_forward(**a)
            got = ssd.recurrence_backward(**a, dy=dy)
            assert bool(y.isfinite().all()), (rv, iv)
            assert all(bool(got[k].isfinite().all()) for k in ("dx", "dr", "di", "ddecay")), (rv, iv)
            if abs(rv) < 60 and abs(iv) < 60:
                want = B.recurrence(x, a["r"], a["i"], decay, grads=(dy, None))
                # below 2^-126 the hardware's exponential gives 0: of what is that small, the
                # input term is off by the root of it, 2^-63 |x|, and its gradient by as much
                for k in ("dx", "di", "dr"):
                    R.check((rv, iv, k), got[k], want[k], want[k + "_err"], 1.0, slack=2.0 ** -58)
                R.check((rv, iv, "y"), y, want["y"], want["y_err"], 1.0, slack=2.0 ** -58)
    # a log-decay of -inf forgets, one of 0 keeps
    z = torch.zeros(1, L, E, device="cuda")
    assert torch.equal(ssd.recurrence_forward(x, z - float("inf")), x)
    R.check("sum", ssd.recurrence_forward(x, z), x.double().cumsum(1).cpu(), x.double().abs().cumsum(1).cpu(), L + B.JOINS)
    g = ssd.recurrence_backward(x, z - float("inf"), None, None, dy)
    assert torch.equal(g["dx"], dy) and bool((g["dr"] == 0).all())


def test_recurrence_nan_stays(ssd):
    """A state that is not a number stays one, across tiles and segments, however much decays."""
    a, r = make(1, 3000, 34, F32, False, False)
    a["r"].fill_(-30.0)
    a["x"][0, 7, 3] = float("nan")
    y, final = ssd.recurrence_forward(**a, return_final_state=True)
    assert bool(y[0, 7:, 3].isnan().all()) and bool(final[0, 3].isnan())
    y[0, :, 3] = 0
    assert bool(y.isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_recurrence_step(ssd, dtype):
    for Bt, E, gated, gate in ((1, 1, True, False), (3, 5, False, True), (70, 130, True, True), (256, 5120, True, True)):
        a, r = make(Bt, 3, E, dtype, gated, gate, 3)
        state = r(Bt, E)
        for t in range(3 if Bt < 200 else 1):
            one = {k: v if v is None or v.dim() == 1 else v[:, t] for k, v in a.items()}
            want = B.recurrence(*[v if v is None or v.dim() == 1 else v[:, t:t + 1] for v in a.values()], state)
            y = ssd.recurrence_step(state, **one)
            R.check((Bt, E, "y"), y, want["y"][:, 0], want["y_err"][:, 0], 1.0)
            R.check((Bt, E, "state"), state, want["final"], want["final_err"], 1.0)


def test_recurrence_differences(ssd):
    """Gradients against differences of the 64-bit form."""
    a, r = make(2, 40, 6, F32, True, True)
    init, dy, dfinal = r(2, 6), r(2, 40, 6), r(2, 6)
    g = ssd.recurrence_backward(**a, dy=dy, init_state=init, dfinal_state=dfinal)
    a = {**{k: v.double().cpu() for k, v in a.items()}, "init": init.double().cpu()}

    def loss(**over):
        o = B.recurrence(**{**a, **over})
        return float((o["y"] * dy.double().cpu()).sum() + (o["final"] * dfinal.double().cpu()).sum())

    h = 1e-5
    for k, at in (("x", (0, 3, 2)), ("r", (1, 20, 5)), ("i", (0, 39, 0)), ("z", (1, 0, 1)), ("decay", (4,)), ("init", (1, 3))):
        d = torch.zeros_like(a[k])
        d[at] = h
        slope = (loss(**{k: a[k] + d}) - loss(**{k: a[k] - d})) / (2 * h)
        # the difference: h^2 of the third derivative and 2^-52 / h of the loss; the gradient: float32
        assert abs(slope - float(g["d" + k][at])) < 1e-4 * max(1.0, abs(slope)), k


def test_recurrence_prompt_then_tokens(ssd):
    """A prompt in one piece, in two pieces and with its last tokens one at a time."""
    for dtype in (BF, F32):
        a, r = make(2, 150, 70, dtype, True, True)
        cut = lambda p, q: {k: v if v.dim() == 1 else v[:, p:q] for k, v in a.items()}  # noqa: E731
        want = B.recurrence(**a)
        y, final = ssd.recurrence_forward(**a, return_final_state=True)
        y1, s = ssd.recurrence_forward(**cut(0, 70), return_final_state=True)
        y2, s = ssd.recurrence_forward(**cut(70, 140), init_state=s, return_final_state=True)
        ys = [y1, y2]
        for t in range(140, 150):
            one = {k: v if v.dim() == 1 else v[:, t] for k, v in a.items()}
            ys.append(ssd.recurrence_step(s, **one)[:, None])
        R.check("pieces", torch.cat(ys, 1), want["y"], want["y_err"], 1.0)
        R.check("final", s, want["final"], want["final_err"], 1.0)
        R.check("whole", final, want["final"], want["final_err"], 1.0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cu", [None, [0, 3, 1300]], ids=["batch", "packed"])
def test_recurrence_growing_states(ssd, cu, dtype):
    """Log-decays above 0, whose products over tiles pass float32 where the state is still (or, going
    back, the gradient) zero: inputs at the last tokens only, gradients of y at the first."""
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    for L, E, rate in ((1300, 40, 0.5), (1300, 33, 1.0), (1300, 200, 8.0)):
        r, few = normal(int(8 * rate)), 6
        x, g, dy = (torch.zeros(1, L, E, dtype=dtype, device="cuda") for _ in range(3))
        g.fill_(rate)
        x[:, -few:], dy[:, :few] = r(1, few, E, dt=dtype), r(1, few, E, dt=dtype)
        want = B.recurrence(x, g, cu=cu, grads=(dy, None))
        y, final, states = ssd.recurrence_forward(x, g, cu_seqlens=c, return_final_state=True, return_states=True)
        check_all((L, rate), dict(y=y, final=final), want, ("y", "final"))
        for s in (states, None):
            got = ssd.recurrence_backward(x, g, None, None, dy, cu_seqlens=c, states=s)
            check_all((L, rate), got, want, ("dx", "dr"))
        # from a state of zero that is given, and a gradient of zero
        if cu is None:
            zero = torch.zeros(1, E, device="cuda")
            assert torch.equal(ssd.recurrence_forward(x, g, init_state=zero), y)
            got = ssd.recurrence_backward(x, g, None, None, dy, init_state=zero, dfinal_state=zero)
            check_all((L, rate), got, want, ("dx", "dr", "dinit"))
