"""A step size that is not a number propagates through the clamp of the
state-space layer (dt_limit) as it does without one, on every path."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
P, LIMIT = 64, (4e-3, 3e-2)


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


def make(Bt, L, H, G, N, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=dtype, sc=1.0: (torch.randn(*s, generator=g) * sc).to(dt).cuda()  # noqa: E731
    dt = (torch.rand(Bt, L, H, generator=g) * 0.05).to(dtype).cuda()
    return dict(x=r(Bt, L, H, P), dt=dt, A=-torch.exp(r(H, dt=F32)), B=r(Bt, L, G, N, sc=N ** -0.5),
                C=r(Bt, L, G, N, sc=N ** -0.5), D=r(H, dt=F32)), r


# (batch, tokens, heads, groups, state): the separate stages, the fused state pass,
# the single-pass kernels uncut and in segments
CASES = [((2, 150, 4, 2, 32), F32, 0), ((2, 150, 4, 2, 32), BF, 0), ((9, 150, 60, 3, 16), BF, 0),
         ((8, 150, 64, 4, 64), BF, 1), ((2, 1500, 8, 2, 128), BF, 2)]


@pytest.mark.parametrize("size,dtype,segments", CASES, ids=str)
def test_forward(ssd, size, dtype, segments):
    a, _ = make(*size, dtype, 1)
    plan = ssd.forward_plan(size[0], size[1], size[2], P, size[3], size[4], 64, dtype)
    assert plan == segments or plan >= segments > 1
    t, h = 70, 1
    a["dt"][0, t, h] = float("nan")
    free, last = ssd.forward(**a, chunk=64, return_final_state=True)
    y, state = ssd.forward(**a, chunk=64, return_final_state=True, dt_limit=LIMIT)
    assert y[0, t:, h].isnan().all() and state[0, h].isnan().all()
    assert torch.equal(y.isnan(), free.isnan()) and torch.equal(state.isnan(), last.isnan())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_step(ssd, dtype):
    a, r = make(3, 1, 4, 2, 64, dtype, 2)
    one = {k: (v[:, 0].contiguous() if k in ("x", "dt", "B", "C") else v) for k, v in a.items()}
    one["dt"][1, 2] = float("nan")
    state = r(3, 4, P, 64, dt=F32)
    y = ssd.step(state, **one, dt_limit=LIMIT)
    bad = torch.zeros(3, 4, dtype=torch.bool)
    bad[1, 2] = True
    assert torch.equal(y.isnan().all(-1).cpu(), bad) and torch.equal(y.isnan().any(-1).cpu(), bad)
    assert torch.equal(state.isnan().flatten(2).all(-1).cpu(), bad)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward(ssd, dtype):
    a, r = make(2, 150, 4, 2, 64, dtype, 3)
    t, h = 70, 1
    a["dt"][0, t, h] = float("nan")
    dy = r(2, 150, 4, P)
    free = ssd.backward(**a, dy=dy)
    got = ssd.backward(**a, dy=dy, dt_limit=LIMIT)
    assert got["ddt"][0, t, h].isnan() and got["dA"][h].isnan()
    for k in got:
        if k != "ddt":  # (outside the bounds ddt is 0 times what comes back)
            assert torch.equal(got[k].isnan(), free[k].isnan()), k
