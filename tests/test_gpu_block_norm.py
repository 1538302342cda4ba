"""The block norm on the GPU against its plain 64-bit form. A norm takes 122 roundings in
32 bits at most (counted in test_gpu_norm.py), the gate 8 + 2 |z|, the scales, dropout and
sum six; backward two norms' statistics and their gradients' sums, the gate twice, and a
rounding per row in sums over rows."""
import pytest
import block_refs as B
import layer_refs as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
OPS = 122
ALPHA, BETA = 1.25, -0.75


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


def make(rows, D, dtype, stream, post, pre, bias, scale, gate, pad, seed=0):
    g = torch.Generator().manual_seed(seed + rows + D)
    r = lambda *s, dt=dtype, sc=1.0, off=0.0: (torch.randn(*s, generator=g) * sc + off).to(dt).cuda()  # noqa: E731
    par = dict(weight=r(D, dt=F32, off=1.0, sc=0.3) if pre else None, bias=r(D, dt=F32) if pre and bias else None,
               post_weight=r(D, dt=F32, off=1.0, sc=0.3) if post else None,
               post_bias=r(D, dt=F32) if post and bias else None, scale=r(D, dt=F32) if scale else None,
               z=r(rows, 2 * D)[:, D:] if gate else None)
    return r(rows, D + pad, off=0.5)[:, pad:], r(rows, D, dt=stream), par, r


# widths below, at and past a vector, a wavefront's vectors, the lanes of a workgroup with one, two and
# four vectors, odd ones, the largest; rows around those of a workgroup and past the grid's
SIZES = [(1, 1), (3, 2), (5, 7), (300, 8), (17, 9), (70, 16), (9, 100), (33, 255), (4, 257), (6, 511), (3, 513), (7, 1000), (5, 1300),
         (2, 2049), (4, 2560), (3, 3001), (2, 4095), (3, 4097), (5, 5119), (2, 8191), (2, 6145), (2, 8192), (2000, 24), (1500, 1000), (1601, 2560)]
# T, stream, rms, post, pre, bias, scale, gate, p, dsum
KINDS = [(BF, F32, True, 1, 1, 0, 1, 0, 0.1, 1), (BF, BF, False, 1, 1, 1, 0, 1, 0.0, 1), (F32, F32, False, 1, 1, 1, 1, 1, 0.5, 0),
         (BF, F32, False, 0, 1, 0, 1, 1, 0.0, 1), (F32, F32, True, 1, 0, 1, 0, 0, 0.25, 1), (BF, BF, True, 0, 1, 1, 0, 0, 0.9, 0),
         (BF, F32, False, 1, 0, 0, 1, 0, 0.0, 1), (F32, F32, False, 0, 1, 0, 0, 0, 0.1, 1), (F32, F32, True, 1, 1, 0, 1, 0, 0.0, 1)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_block_norm(ssd, size):
    rows, D = size
    rng, eps = (11, 12), 1e-5
    for n, (dtype, stream, rms, post, pre, bias, scale, gate, p, skip) in enumerate(KINDS):
        name = (size, n)
        x, res, par, r = make(rows, D, dtype, stream, post, pre, bias, scale, gate, (3, 0, 8)[n % 3], n)
        kw = dict(residual_scale=ALPHA, branch_scale=BETA, p=p, rng=rng)
        ref = B.Block(x, res, *par.values(), ALPHA, BETA, p, rng, eps, rms)
        kz = 8 + 2 * float(par["z"].abs().max()) if gate else 0
        y, total, stats = ssd.block_norm_forward(x, res, **par, **kw, eps=eps, rms=rms, return_stats=True)
        assert total.dtype == stream
        R.check((name, "sum"), total, ref.total, ref.total_mag, OPS + kz + 6)
        if pre:
            want, mag = ref.y(total)
            R.check((name, "y"), y, want, mag, OPS)
        else:
            assert y is None
        y2, total2 = ssd.block_norm_forward(x, res, **par, **kw, eps=eps, rms=rms)
        assert torch.equal(total, total2) and (not pre or torch.equal(y, y2))
        dy, dsum = r(rows, D) if pre else None, r(rows, D, dt=stream) if skip else None
        got = ssd.block_norm_backward(dy, dsum, x, total, stats, **par, **kw)
        want, mag = ref.grads(dy, dsum, total)
        assert {k for k in got if got[k] is not None} == set(want)
        for k in want:
            many = rows if k not in ("dx", "dresidual", "dz") else 0
            R.check((name, k), got[k], want[k], mag[k], 4 * OPS + 2 * kz + 16 + many)
        again = ssd.block_norm_backward(dy, dsum, x, total, stats, **par, **kw)
        assert all(torch.equal(got[k], again[k]) for k in want)


def test_block_norm_mask_is_dropouts(ssd):
    """The same elements as ``dropout`` drops, of rows in the order of the leading axes."""
    x = torch.randn(3, 50, 333, device="cuda")
    w = torch.ones(333, device="cuda")
    _, total = ssd.block_norm_forward(x, torch.zeros_like(x), w, p=0.4, rng=(5, 6))
    assert torch.equal(total, ssd.dropout(x, 0.4, (5, 6)))
    _, total = ssd.block_norm_forward(x, torch.ones_like(x), w, p=1.0, rng=(5, 6), residual_scale=0.5)
    assert bool((total == 0.5).all())


def test_block_norm_special_rows(ssd):
    """Constant rows have no deviation, rows of zeros stay zero, NaN stays in its row, and what
    is dropped is dropped whatever it is (without a norm in front)."""
    D = 512
    x = torch.zeros(4, D, device="cuda")
    x[0], x[2, 5] = 3.0, float("nan")
    one, quarter = torch.ones(D, device="cuda"), torch.full((D,), 0.25, device="cuda")
    y, total = ssd.block_norm_forward(x, torch.zeros_like(x), one, quarter, one, quarter)
    assert bool((total[[0, 1, 3]] == 0.25).all()) and bool((y[[0, 1, 3]] == 0.25).all())
    assert bool(total[2].isnan().all()) and bool(y[2].isnan().all())
    rng = (1, 2)
    keep = B.kept(4, D, 0.5, *rng).cuda()
    x = torch.where(keep, 1.0, float("inf"))
    _, total = ssd.block_norm_forward(x, torch.ones_like(x), one, p=0.5, rng=rng)
    assert torch.equal(total, torch.where(keep, 3.0, 1.0))
    # and in the gradient that reaches the block
    _, total, stats = ssd.block_norm_forward(torch.ones_like(x), torch.ones_like(x), one, p=0.5, rng=rng, return_stats=True)
    g = ssd.block_norm_backward(torch.zeros_like(x), torch.where(keep, 1.0, float("nan")), torch.ones_like(x), total, stats, one,
                                p=0.5, rng=rng)
    assert torch.equal(g["dx"], torch.where(keep, 2.0, 0.0)) and torch.equal(g["dresidual"].isnan(), ~keep)


def test_block_norm_shapes_and_differences(ssd):
    """Leading axes of any number; gradients against differences of the 64-bit form."""
    for rms in (False, True):
        x, res, par, r = make(6, 40, F32, F32, 1, 1, 1, 1, 1, 0)
        x, res, par["z"] = x.view(2, 3, 40), res.view(2, 3, 40), par["z"].contiguous().view(2, 3, 40)
        kw = dict(residual_scale=ALPHA, branch_scale=BETA, p=0.3, rng=(3, 4))
        y, total, stats = ssd.block_norm_forward(x, res, **par, **kw, rms=rms, return_stats=True)
        assert y.shape == total.shape == x.shape and stats[1].shape == (2, 3)
        dy, dsum = r(2, 3, 40), r(2, 3, 40)
        g = ssd.block_norm_backward(dy, dsum, x, total, stats, **par, **kw)
        t = {k: v.double().cpu() for k, v in dict(x=x, residual=res, **par).items()}

        def loss(**over):
            ref = B.Block(**{**t, **over}, alpha=ALPHA, beta=BETA, p=0.3, rng=(3, 4), rms=rms)
            return float((ref.y(ref.total)[0] * dy.double().cpu()).sum() + (ref.total * dsum.double().cpu()).sum())

        h = 1e-5
        for k, at in (("x", (1, 2, 7)), ("residual", (0, 1, 39)), ("z", (1, 0, 3)), ("weight", (5,)), ("bias", (6,)),
                      ("post_weight", (7,)), ("post_bias", (8,)), ("scale", (9,))):
            d = torch.zeros_like(t[k])
            d[at] = h
            slope = (loss(**{k: t[k] + d}) - loss(**{k: t[k] - d})) / (2 * h)
            assert abs(slope - float(g["d" + k][at])) < 1e-4 * max(1.0, abs(slope)), (rms, k)


def test_block_norm_far_rows(ssd):
    """Rows of x and z whose offsets pass 2^32 elements."""
    rows, D, row = 300, 40, (1 << 24) - 8
    far = torch.empty((rows - 1) * row + D, dtype=BF, device="cuda").as_strided((rows, D), (row, 1))
    x, res, par, r = make(rows, D, BF, F32, 1, 1, 0, 1, 1, 0)
    z, dy = par.pop("z"), r(rows, D)
    far.copy_(x)
    y, total, stats = ssd.block_norm_forward(x, res, **par, z=x, return_stats=True)
    yf, tf, _ = ssd.block_norm_forward(far, res, **par, z=far, return_stats=True)
    assert torch.equal(y, yf) and torch.equal(total, tf)
    a = ssd.block_norm_backward(dy, res, x, total, stats, **par, z=x)
    b = ssd.block_norm_backward(dy, res, far, total, stats, **par, z=far)
    assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")], ids=["inf", "nan"])
@pytest.mark.parametrize("kind", [(BF, F32, True, 0, 0), (BF, F32, False, 1, 1), (F32, F32, False, 0, 1), (BF, BF, True, 0, 1)],
                         ids=str)
def test_block_norm_dropped_values(ssd, kind, bad):
    """What x (without a norm in front) and the gate hold where an element is dropped reaches no
    result and no gradient: the same bits as with zeros there."""
    dtype, stream, rms, post, gate = kind
    for rows, D, p in ((300, 8, 0.5), (7, 1000, 0.1), (5, 2560, 0.9), (3, 8192, 1.0)):
        x, res, par, r = make(rows, D, dtype, stream, post, 1, not rms, 1, gate, 0)
        kw = dict(p=p, rng=(5, 6))
        lost = ~B.kept(rows, D, p, 5, 6).cuda()
        dy, dsum = r(rows, D), r(rows, D, dt=stream)
        out = []
        for fill in (0.0, bad):
            tx = x if post else x.masked_fill(lost, fill)
            q = dict(par, z=par["z"].masked_fill(lost, fill)) if gate else par
            y, total, stats = ssd.block_norm_forward(tx, res, **q, **kw, rms=rms, return_stats=True)
            out.append({**ssd.block_norm_backward(dy, dsum, tx, total, stats, **q, **kw), "y": y, "sum": total})
        for k, t in out[0].items():
            assert t is None or torch.equal(out[1][k], t) and bool(t.isfinite().all()), (rows, D, k)
