"""The normalisation on the GPU against its plain 64-bit form.

Roundings in 32 bits: a row's sum takes at most V NV + 6 + 16 additions one
after another (values of a lane, lanes of a wavefront, wavefronts), below 56 at
16384 values; the mean, then the deviations, their squares' sum, the square
root and the quotient, the products with weight and bias: 2 * 56 + 10. The
gate's SiLU adds 8 + 2 |z|. Gradients run through the two sums once more. Sums
over rows add a rounding per row."""
import pytest
import layer_refs as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
OPS = 2 * 56 + 10


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


def make(rows, D, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=dtype, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt).cuda()  # noqa: E731
    x = r(rows, D + pad, off=0.5)[:, pad:]
    return x, r(D, dt=F32, off=1.0, sc=0.3), r(D, dt=F32), r


# widths below, at and past a vector, a wavefront's vectors (512 / 256 values), a
# workgroup's (8192 / 4096), odd ones, the largest; rows around those of a workgroup
SIZES = [(1, 1), (3, 2), (5, 7), (300, 8), (17, 9), (70, 16), (9, 100), (33, 255), (4, 257), (6, 511),
         (3, 513), (7, 1000), (2, 4097), (5, 5119), (3, 8193), (2, 16383), (2, 16384)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_norm(ssd, size, dtype):
    rows, D = size
    for rms, bias, pad in ((False, True, 0), (True, False, 5), (False, False, 8)):
        x, w, b, r = make(rows, D, dtype, D, pad)
        b = b if bias else None
        y, mean, rstd = ssd.norm_forward(x, w, b, eps=EPS, rms=rms, return_stats=True)
        want, m, s, mag = R.norm(x, w, b, rms, EPS)
        R.check((size, rms, "y"), y, want, mag, OPS)
        R.check((size, rms, "rstd"), rstd, s, s + s ** 3 * x.double().cpu().abs().mean(-1) ** 2, OPS)
        if rms:
            assert mean is None
        else:
            R.check((size, "mean"), mean, m, x.double().cpu().abs().mean(-1), 60)
        dy = r(rows, D)
        got = ssd.norm_backward(dy, x, w, mean, rstd)
        want, mag = R.norm_grads(dy, x, w, rms, EPS)
        for k in ("dx", "dweight", "dbias"):
            if k == "dbias" and rms:
                assert got[k] is None
                continue
            R.check((size, rms, k), got[k], want[k], mag[k], 2 * OPS + (rows if k != "dx" else 0))


@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("size", [(3, 5), (40, 64), (7, 513), (5, 2560), (2, 12000)], ids=str)
def test_norm_residual(ssd, size, dtype, stream):
    rows, D = size
    for rms in (False, True):
        x, w, b, r = make(rows, D, dtype, D, 3)
        res, dy, dres = r(rows, D, dt=stream), r(rows, D), r(rows, D, dt=stream)
        y, total, mean, rstd = ssd.norm_forward(x, w, b, residual=res, eps=EPS, rms=rms, return_stats=True)
        exact = x.double().cpu() + res.double().cpu()
        R.check((size, "sum"), total, exact, exact.abs(), 1)
        want, _, _, mag = R.norm(total, w, b, rms, EPS)  # the norm reads the sum as it is kept
        R.check((size, "y"), y, want, mag, OPS)
        got = ssd.norm_backward(dy, total, w, mean, rstd, dresidual=dres)
        want, mag = R.norm_grads(dy, total, w, rms, EPS, dres=dres)
        assert got["dx"].dtype == dtype and got["dresidual"].dtype == stream
        R.check((size, "dx"), got["dx"], want["dx"], mag["dx"], 2 * OPS)
        R.check((size, "dres"), got["dresidual"], want["dx"], mag["dx"], 2 * OPS)
        R.check((size, "dw"), got["dweight"], want["dweight"], mag["dweight"], 2 * OPS + rows)
        if not rms:
            R.check((size, "db"), got["dbias"], want["dbias"], mag["dbias"], rows)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [(3, 5), (40, 64), (7, 513), (5, 5120), (2, 12001)], ids=str)
def test_norm_gated(ssd, size, dtype):
    rows, D = size
    for rms in (True, False):
        x, w, b, r = make(rows, D, dtype, D + 1)
        z, dy = r(rows, 2 * D)[:, :D], r(rows, D)
        y, mean, rstd = ssd.norm_forward(x, w, b, z=z, eps=EPS, rms=rms, return_stats=True)
        want, _, _, mag = R.norm(x, w, b, rms, EPS, z)
        gate = 2 * (8 + 2 * float(z.abs().max()))
        # |silu(z)| can be far below the magnitudes |x| |z| that its rounding is relative to
        R.check((size, "y"), y, want, mag, OPS + gate)
        got = ssd.norm_backward(dy, x, w, mean, rstd, z=z)
        want, mag = R.norm_grads(dy, x, w, rms, EPS, z)
        for k in ("dx", "dz", "dweight") + (() if rms else ("dbias",)):
            R.check((size, rms, k), got[k], want[k], mag[k], 2 * (OPS + gate) + (rows if k[1] in "wb" else 0))


def test_norm_many_rows(ssd):
    """More rows than the grid holds at once, short and long ones; the weight's
    gradient is the same on every call."""
    for rows, D in ((20011, 24), (5003, 1000)):
        x, w, b, r = make(rows, D, BF, 1)
        dy = r(rows, D)
        y, mean, rstd = ssd.norm_forward(x, w, b, eps=EPS, return_stats=True)
        want, _, _, mag = R.norm(x, w, b, False, EPS)
        R.check("y", y, want, mag, OPS)
        got = ssd.norm_backward(dy, x, w, mean, rstd)
        want, mag = R.norm_grads(dy, x, w, False, EPS)
        for k in ("dx", "dweight", "dbias"):
            R.check((rows, k), got[k], want[k], mag[k], 2 * OPS + (rows if k != "dx" else 0))
        again = ssd.norm_backward(dy, x, w, mean, rstd)
        assert all(torch.equal(got[k], again[k]) for k in ("dx", "dweight", "dbias"))


def test_norm_special_rows(ssd):
    """A constant row has no deviation (y = bias exactly where the mean is exact),
    a row far from zero keeps its small deviations, NaN stays in its row."""
    D = 512
    x = torch.zeros(4, D, device="cuda")
    x[0] = 3.0
    x[1] = 4096.0 + torch.arange(D, device="cuda") / 512
    x[2, 5] = float("nan")
    w, b = torch.ones(D, device="cuda"), torch.full((D,), 0.25, device="cuda")
    y = ssd.norm_forward(x, w, b, eps=EPS).cpu()
    assert (y[0] == 0.25).all() and (y[3] == 0.25).all() and y[2].isnan().all()
    want, _, _, _ = R.norm(x[1:2], w, b, False, EPS)
    # the row's values need 22 bits: sums round by half of 2^-2 at 2^21; the mean by 2^-13
    assert float((y[1].double() - want[0]).abs().max()) < 2.0 ** -12 * 4


def test_norm_shapes_and_differences(ssd):
    x = torch.randn(2, 3, 40, device="cuda")
    w = torch.rand(40, device="cuda") + 0.5
    b = torch.randn(40, device="cuda")
    dy = torch.randn_like(x)
    y, mean, rstd = ssd.norm_forward(x, w, b, return_stats=True)
    assert y.shape == x.shape and mean.shape == rstd.shape == (2, 3)
    got = ssd.norm_backward(dy, x, w, mean, rstd)
    f = lambda xx, ww: (R.norm(xx, ww, b, False, 1e-5)[0] * dy.double().cpu()).sum()  # noqa: E731
    h = 1e-4
    for grad, at in (("dx", (1, 2, 7)), ("dx", (0, 0, 39)), ("dweight", (11,))):
        t = x if grad == "dx" else w
        d = torch.zeros(t.shape, dtype=torch.float64)
        d[at] = h
        t64 = t.double().cpu()
        if grad == "dx":
            slope = float(f(t64 + d, w) - f(t64 - d, w)) / (2 * h)
        else:
            slope = float(f(x, t64 + d) - f(x, t64 - d)) / (2 * h)
        assert abs(slope - float(got[grad][at])) < 1e-4 * max(1.0, abs(slope))


def test_norm_captured(ssd):
    x, w, b, r = make(60, 700, BF, 3)
    dy, res = r(60, 700), r(60, 700, dt=F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, total, mean, rstd = ssd.norm_forward(x, w, b, residual=res, return_stats=True)
        ssd.norm_backward(dy, total, w, mean, rstd, dresidual=res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, total, mean, rstd = ssd.norm_forward(x, w, b, residual=res, return_stats=True)
        grads = ssd.norm_backward(dy, total, w, mean, rstd, dresidual=res)
    for k in range(4):
        x.copy_(torch.randn(x.shape).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        ey, et, em, er = ssd.norm_forward(x, w, b, residual=res, return_stats=True)
        eg = ssd.norm_backward(dy, et, w, em, er, dresidual=res)
        assert torch.equal(y, ey) and torch.equal(total, et)
        assert all(torch.equal(grads[n], eg[n]) for n in eg)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [(40, 24), (7, 513), (5, 2560), (2, 12000)], ids=str)
def test_norm_rms_bias_gradient(ssd, size, dtype):
    """The root-mean-square form takes a bias too; its gradient on request. A
    sum over rows adds at most a rounding per row of its terms."""
    rows, D = size
    x, w, b, r = make(rows, D, dtype, D, 3)
    y, mean, rstd = ssd.norm_forward(x, w, b, eps=EPS, rms=True, return_stats=True)
    want, _, _, mag = R.norm(x, w, b, True, EPS)
    R.check((size, "y"), y, want, mag, OPS)
    dy = r(rows, D)
    plain = ssd.norm_backward(dy, x, w, mean, rstd)
    got = ssd.norm_backward(dy, x, w, mean, rstd, want_dbias=True)
    assert plain["dbias"] is None and all(torch.equal(plain[k], got[k]) for k in ("dx", "dweight"))
    want, mag = R.norm_grads(dy, x, w, True, EPS)
    R.check((size, "dbias"), got["dbias"], want["dbias"], mag["dbias"], rows)
    h = 1e-3  # y is linear in the bias: a difference is exact up to 64-bit rounding
    step = torch.zeros(D, dtype=torch.float64)
    step[D - 1] = h
    f = lambda bb: (R.norm(x, w, bb, True, EPS)[0] * dy.double().cpu()).sum()  # noqa: E731
    slope = float(f(b.double().cpu() + step) - f(b.double().cpu() - step)) / (2 * h)
    assert abs(slope - float(got["dbias"][D - 1])) < 1e-4 * max(1.0, abs(slope))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [(40, 24), (7, 513), (2, 12000)], ids=str)
def test_norm_without_bias_gradient(ssd, size, dtype):
    """A layer norm without a bias asks for no gradient of it, and the other
    gradients are the same."""
    rows, D = size
    x, w, _, r = make(rows, D, dtype, D)
    _, mean, rstd = ssd.norm_forward(x, w, eps=EPS, return_stats=True)
    dy = r(rows, D)
    whole = ssd.norm_backward(dy, x, w, mean, rstd)
    got = ssd.norm_backward(dy, x, w, mean, rstd, want_dbias=False)
    assert got["dbias"] is None and whole["dbias"] is not None
    assert all(torch.equal(got[k], whole[k]) for k in ("dx", "dweight"))
    from structured_state_space_ssd_amd._native import lib
    need = lib.ssd_norm_backward_workspace_size(rows, D, int(dtype == BF), 0)
    again = ssd.norm_backward(dy, x, w, mean, rstd, want_dbias=False,
                              workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(again["dweight"], got["dweight"])


@pytest.mark.parametrize("dtype,stream", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("size", [(40, 24), (5, 2560), (2, 12000)], ids=str)
def test_norm_residual_without_skip(ssd, size, dtype, stream):
    """After the last norm nothing comes back by the skip connection: the
    stream's gradient is the norm's alone, in the stream's own type."""
    rows, D = size
    x, w, b, r = make(rows, D, dtype, D)
    res, dy = r(rows, D, dt=stream), r(rows, D)
    _, total, mean, rstd = ssd.norm_forward(x, w, b, residual=res, eps=EPS, return_stats=True)
    got = ssd.norm_backward(dy, total, w, mean, rstd, want_dresidual=True)
    plain = ssd.norm_backward(dy, total, w, mean, rstd)
    assert "dresidual" not in plain and torch.equal(plain["dx"], got["dx"])
    want, mag = R.norm_grads(dy, total, w, False, EPS)
    assert got["dresidual"].dtype == stream and got["dx"].dtype == dtype
    R.check((size, "dresidual"), got["dresidual"], want["dx"], mag["dx"], 2 * OPS)
    assert torch.equal(got["dx"], got["dresidual"].to(dtype))
    # a skip gradient may also reach the sum while only x needs a gradient
    dres = r(rows, D, dt=stream)
    both = ssd.norm_backward(dy, total, w, mean, rstd, dresidual=dres)
    one = ssd.norm_backward(dy, total, w, mean, rstd, dresidual=dres, want_dresidual=False)
    assert "dresidual" not in one and torch.equal(one["dx"], both["dx"])


# ---- exact sums -------------------------------------------------------------
# The statistics are inputs of the backward: with whole-number means and a power of
# two for rstd, n = (u - m) r and its products with whole-number gradients are small
# integers, so that the sums over rows are exact in any order and compared for equality.
# The gradients are positive, so that every row moves dbias.

def blocks_of(rows, D, dtype, want_db=True):
    """Workgroups of a backward call, by its workspace."""
    from structured_state_space_ssd_amd._native import lib
    return lib.ssd_norm_backward_workspace_size(rows, D, int(dtype == BF), int(want_db)) // (4 * D * (1 + want_db))


def check_exact_sums(ssd, rows, D, dtype, rms, gate, stream=None):
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    r = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda")  # noqa: E731
    x, dy, mean = r(-3, 3, rows, D), r(1, 3, rows, D), r(-2, 2, rows)
    w = torch.ones(D, device="cuda")
    m = None if rms else mean.float()
    scale, z = 1.0, None
    if gate:  # silu(128) = 128 in float32: u = 128 x
        z, scale = torch.full((rows, D), 128.0, dtype=dtype, device="cuda"), 128.0
        m = None if rms else m * scale
    # (rows differ in rstd, so that a row taken with another's statistics shows)
    power = r(0, 2, rows)
    rstd = 2.0 ** power.float() / scale
    got = ssd.norm_backward(dy.to(dtype), x.to(stream or dtype), w, m, rstd, z=z, want_dbias=True)
    # n = (x - m) 2^power, at most 20 of them and dy 3 to a row: exact to 2^24 / 60 rows
    assert rows * 60 < 1 << 24
    n = (x.double() - (0 if rms else mean.double()[:, None])) * 2.0 ** power.double()[:, None]
    assert torch.equal(got["dweight"].double(), (dy * n).sum(0)), "dweight"
    assert torch.equal(got["dbias"].double(), dy.double().sum(0)), "dbias"


# (rows, width): more short rows than the grid's lanes hold at once, so that groups of
# 1 to 64 lanes of a wavefront take several each and some one less; and long rows, one
# or several vectors to a lane
MANY = [(270001, 8), (140003, 16), (70005, 24), (140001, 33), (9001, 256), (9003, 512), (5003, 1000),
        (2050, 2560), (1031, 8200), (777, 16384)]


# (a gated x has the gate's type)
@pytest.mark.parametrize("dtype,stream,gate", [(BF, BF, False), (BF, F32, False), (F32, F32, False), (BF, BF, True),
                                               (F32, F32, True)],
                         ids=["bf16", "bf16_f32", "f32", "bf16_gated", "f32_gated"])
@pytest.mark.parametrize("size", MANY, ids=str)
def test_norm_row_sums_exact(ssd, size, dtype, stream, gate):
    rows, D = size
    V = 8 if dtype == BF else 4
    vectors, lanes = -(-D // V), 1
    while lanes < min(vectors, 64):
        lanes *= 2
    groups = 256 // lanes if vectors <= 64 else 1
    assert blocks_of(rows, D, dtype) * groups < rows  # a group takes more than one row
    for rms in (False, True):
        check_exact_sums(ssd, rows, D, dtype, rms, gate, stream)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("size", [(200003, 16), (100005, 24), (13001, 256), (9003, 512)], ids=str)
def test_norm_many_short_rows(ssd, size, dtype, gate):
    """y, statistics, dx and dz of more short rows than the grid holds, forward too
    (1536 lanes to a CU: 6 workgroups of 256)."""
    rows, D = size
    V = 8 if dtype == BF else 4
    assert rows * 2 ** (-(-D // V) - 1).bit_length() > 256 * 6 * 256
    for rms in (False, True):
        x, w, b, r = make(rows, D, dtype, D)
        z, dy = (r(rows, D), r(rows, D)) if gate else (None, r(rows, D))
        y, mean, rstd = ssd.norm_forward(x, w, b, z=z, eps=EPS, rms=rms, return_stats=True)
        want, m, s, mag = R.norm(x, w, b, rms, EPS, z)
        extra = 2 * (8 + 2 * float(z.abs().max())) if gate else 0
        R.check((size, rms, "y"), y, want, mag, OPS + extra)
        got = ssd.norm_backward(dy, x, w, mean, rstd, z=z)
        want, mag = R.norm_grads(dy, x, w, rms, EPS, z)
        for k in ("dx", "dz") if gate else ("dx",):
            R.check((size, rms, k), got[k], want[k], mag[k], 2 * (OPS + extra))
