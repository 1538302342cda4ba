"""The short causal convolution on the GPU against its plain 64-bit form.

Roundings in 32 bits: W + 1 for v, then sigmoid(v): its exponent's rounding
(2 |v| U32 of e^-v, itself at most the quotient), exponential and reciprocal 2
each, sum and product 1 each. A SiLU multiplies v's error by at most 1.1. A sum
over n tokens adds at most n roundings of its terms' magnitudes."""
import pytest
import layer_refs as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


def make(Bt, L, K, W, dtype, seed, pad=0, init=False, bias=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(Bt, L, K + pad, generator=g) * scale).to(dtype).cuda()[..., pad:]
    w = torch.randn(K, W, generator=g).cuda()
    b = torch.randn(K, generator=g).cuda() if bias else None
    i = torch.randn(Bt, W - 1, K, generator=g).to(dtype).cuda() if init else None
    return x, w, b, i, g


def check_y(name, y, x, w, b, act, init=None, cu=None):
    v, want, final, mag = R.conv(x, w, b, act, init, cu)
    W = w.shape[1]
    # v's error, and the activation's own: relative to |v|, its exponent's part grows with |v|
    total = 1.1 * (W + 1) * mag + (want.abs() * (8 + 2 * v.abs()) if act else 0)
    R.check(name, y, want, total, 1.0)
    return final


# lengths around the tile (16 and 8 tokens) and the 8 rows fetched at a time, shorter
# than the filter, one token; channels below, at and past a vector, odd ones
SIZES = [(1, 1, 1), (2, 1, 16), (1, 2, 7), (3, 3, 8), (2, 9, 33), (1, 31, 64), (2, 32, 5),
         (1, 33, 100), (2, 65, 17), (1, 257, 40), (1, 100, 1025)]


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_conv_forward(ssd, size, dtype, W):
    Bt, L, K = size
    for act, init, bias, pad in ((True, False, True, 0), (True, True, True, 3), (False, True, False, 8)):
        x, w, b, i, _ = make(Bt, L, K, W, dtype, 7 * L + K + W, pad, init, bias)
        y, final = ssd.conv_forward(x, w, b, silu=act, init_state=i, return_final_state=True)
        want = check_y((size, W, act), y, x, w, b, act, i)
        assert torch.equal(final.double().cpu(), want)
        assert torch.equal(ssd.conv_forward(x, w, b, silu=act, init_state=i), y)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("split", [(8, 8, 8), (17, 3, 5), (1, 1), (64, 16, 16), (30,), (1000, 9, 9)], ids=str)
def test_conv_forward_split(ssd, split, dtype):
    x, w, b, i, _ = make(2, 21, sum(split), 4, dtype, sum(split), 5, True)
    whole = ssd.conv_forward(x, w, b, init_state=i)
    parts = ssd.conv_forward(x, w, b, init_state=i, split=split)
    assert isinstance(parts, tuple) and all(p.is_contiguous() for p in parts)
    assert torch.equal(torch.cat(parts, -1), whole)


PACKED = [[0, 1], [0, 5, 5, 6, 40], [0, 0, 0, 33], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 70],
          [0, 31, 32, 64, 96, 99, 99], [0, 2, 200], list(range(0, 301, 3))]


@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cu", PACKED, ids=lambda c: f"{len(c) - 1}seq{c[-1]}")
def test_conv_packed(ssd, cu, dtype, W):
    x, w, b, _, _ = make(1, cu[-1], 24, W, dtype, cu[-1], 2)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, final = ssd.conv_forward(x, w, b, return_final_state=True, cu_seqlens=c)
    want = check_y(cu, y, x, w, b, True, None, cu)
    assert torch.equal(final.double().cpu(), want)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_conv_backward(ssd, size, dtype, W):
    Bt, L, K = size
    for act, init, fin, pad in ((True, False, False, 0), (True, True, True, 3), (False, True, False, 8)):
        x, w, b, i, g = make(Bt, L, K, W, dtype, 7 * L + K + W, pad, init)
        dy = torch.randn(Bt, L, K, generator=g).to(dtype).cuda()
        df = torch.randn(Bt, W - 1, K, generator=g).to(dtype).cuda() if fin else None
        got = ssd.conv_backward(x, w, b, dy, silu=act, init_state=i, dfinal_state=df)
        want, mag = R.conv_grads(x, w, b, act, dy, i, df)
        # g: v's W + 1 roundings through a second derivative of at most 1/2 times its
        # magnitude, and the derivative's own; then W more products and sums
        vmag = float(R.conv(x, w, b, act, i)[3].max())
        ops = W + 14 + (W + 1) * vmag
        for k in ("dx", "dinit", "dweight", "dbias"):
            if got[k] is None:
                assert k == "dinit" and i is None
                continue
            n = Bt * L if k in ("dweight", "dbias") else 0
            R.check((size, k, act), got[k], want[k], mag[k], ops + n)


def test_conv_backward_many_tiles(ssd):
    """Few channels over many tokens: more partial rows than one pass sums up."""
    Bt, L, K, W = 3, 8000, 5, 3
    x, w, b, _, g = make(Bt, L, K, W, F32, 77)
    dy = torch.randn(Bt, L, K, generator=g).cuda()
    got = ssd.conv_backward(x, w, b, dy)
    want, mag = R.conv_grads(x, w, b, True, dy)
    ops = W + 14 + (W + 1) * float(R.conv(x, w, b, True)[3].max())
    for k in ("dx", "dweight", "dbias"):
        R.check(k, got[k], want[k], mag[k], ops + (Bt * L if k != "dx" else 0))


def test_conv_backward_split_and_differences(ssd):
    """dy in parts gives the same as whole; the gradient is the loss's slope:
    a central difference of the 64-bit form with step h is off by h^2 / 6 times
    the third derivative (h = 1e-4: below 1e-6 here)."""
    split = (17, 3, 5)
    x, w, b, i, g = make(2, 13, 25, 4, F32, 3, 0, True)
    dy = torch.randn(2, 13, 25, generator=g).cuda()
    whole = ssd.conv_backward(x, w, b, dy, init_state=i)
    parts = ssd.conv_backward(x, w, b, tuple(p.contiguous() for p in dy.split(split, -1)), init_state=i)
    for k in whole:
        assert torch.equal(whole[k], parts[k]), k

    def loss(**kw):
        a = dict(x=x, weight=w, bias=b, init=i)
        a = {k: v.double().cpu() for k, v in a.items()}
        a.update(kw)
        return (R.conv(a["x"], a["weight"], a["bias"], True, a["init"])[1] * dy.double().cpu()).sum()

    h = 1e-4
    for key, grad, t, at in (("x", "dx", x, (1, 4, 7)), ("weight", "dweight", w, (3, 1)),
                             ("bias", "dbias", b, (24,)), ("init", "dinit", i, (0, 2, 9))):
        d = torch.zeros_like(t, dtype=torch.float64, device="cpu")
        d[at] = h
        t64 = t.double().cpu()
        slope = float(loss(**{key: t64 + d}) - loss(**{key: t64 - d})) / (2 * h)
        assert abs(slope - float(whole[grad][at])) < 1e-4 * max(1.0, abs(slope)), key


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("split", [None, (9, 3, 5)], ids=str)
def test_conv_step_goes_on(ssd, split, W, dtype):
    """Prompt, then token by token: the same as the whole sequence at once, bit
    for bit (both add the taps in the same order)."""
    Bt, L, K = 5, 12, 17
    x, w, b, _, _ = make(Bt, L, K, W, dtype, W, 4)
    whole = ssd.conv_forward(x, w, b)
    for start in (1, 2, 7):
        y, state = ssd.conv_forward(x[:, :start], w, b, return_final_state=True)
        assert torch.equal(y, whole[:, :start])
        for t in range(start, L):
            y = ssd.conv_step(state, x[:, t], w, b, split=split)
            y = torch.cat(y, -1) if split else y
            assert torch.equal(y, whole[:, t]), (start, t)
        assert torch.equal(state, x[:, L - (W - 1):])


def test_conv_values_at_the_ends(ssd):
    """Infinities and NaN reach only the tokens whose window holds them, and
    only their own channels; large negative v gives 0, not NaN. A gradient past
    the sequence's end stays out of it."""
    x = torch.zeros(1, 40, 9, device="cuda")
    x[0, 10, 2], x[0, 20, 3], x[0, 39, 4] = float("nan"), float("inf"), float("inf")
    x[0, :, 5] = -1e4
    w, b = torch.ones(9, 4, device="cuda"), torch.zeros(9, device="cuda")
    y = ssd.conv_forward(x, w, b).cpu()[0]
    assert y[10:14, 2].isnan().all() and (y[20:24, 3] == float("inf")).all() and y[39, 4] == float("inf")
    keep = torch.ones(40, 9, dtype=torch.bool)
    keep[10:14, 2] = keep[20:24, 3] = keep[39, 4] = False
    assert (y[keep] == 0).all()
    dx = ssd.conv_backward(x, w, b, torch.ones_like(x))["dx"].cpu()[0]
    assert dx[:, [0, 1, 6, 7, 8]].isfinite().all() and dx[38, 0] == 1.0 and dx[39, 0] == 0.5


def test_conv_captured(ssd):
    """Captured once, replayed with other inputs in the same memory, with eager
    calls and synchronisations between."""
    x, w, b, i, g = make(2, 50, 24, 4, BF, 5, 0, True)
    dy = torch.randn(2, 50, 24, generator=g).to(BF).cuda()
    state = i.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssd.conv_backward(x, w, b, dy, init_state=i)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, fin = ssd.conv_forward(x, w, b, init_state=i, return_final_state=True)
        grads = ssd.conv_backward(x, w, b, dy, init_state=i)
        ys = ssd.conv_step(state, x[:, 0], w, b)
    for k in range(4):
        x.copy_(torch.randn(x.shape, generator=g).to(BF))
        state.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        ey, efin = ssd.conv_forward(x, w, b, init_state=i, return_final_state=True)
        eg = ssd.conv_backward(x, w, b, dy, init_state=i)
        st = i.clone()
        es = ssd.conv_step(st, x[:, 0], w, b)
        assert torch.equal(y, ey) and torch.equal(fin, efin) and torch.equal(ys, es)
        assert torch.equal(state, st) and all(torch.equal(grads[n], eg[n]) for n in eg)


# ---- exact sums -------------------------------------------------------------
# Small integers in float32, without the activation: every product and every
# partial sum is a whole number below 2^24 and so exact in any order, and each
# result is compared for equality. All gradients are positive, so that every
# token moves dbias: a partial row left out or added twice changes it.

def integers(Bt, L, K, W, seed, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda")  # noqa: E731
    return (r(-3, 3, Bt, L, K).to(dtype), r(-2, 2, K, W).float(), r(-3, 3, K).float(),
            r(-3, 3, Bt, W - 1, K).to(dtype), r(1, 3, Bt, L, K).to(dtype), r(-3, 3, Bt, W - 1, K).to(dtype))


def exact_forward(x, w, b, init=None, cu=None):
    """y and the final states in float64, which holds every value exactly."""
    Bt, L, K = x.shape
    W = w.shape[1]
    x, w = x.double(), w.double()
    head = x.new_zeros(Bt, W - 1, K) if init is None else init.double()
    xs = torch.cat([head, x], 1)
    y = b.double().expand(Bt, L, K).clone()
    since = None
    if cu is not None:  # tokens of the same sequence before each one
        at = torch.arange(L, device=x.device)
        c = torch.tensor(cu, device=x.device)
        since = at - c[torch.searchsorted(c, at, right=True) - 1]
    for k in range(W):
        term = w[:, k] * xs[:, k:k + L]
        y += term if since is None else term * (since >= W - 1 - k)[:, None]
    if cu is None:
        return y, xs[:, L:]
    c = torch.tensor(cu, device=x.device)
    rows = c[1:, None] - (W - 1) + torch.arange(W - 1, device=x.device)
    return y, torch.where((rows >= c[:-1, None])[..., None], x[0][rows.clamp(min=0)], 0.0)


def exact_backward(x, w, dy, init, dfinal):
    Bt, L, K = x.shape
    W = w.shape[1]
    head = x.new_zeros(Bt, W - 1, K) if init is None else init
    xs, dy, w = torch.cat([head, x], 1).double(), dy.double(), w.double()
    dxs = torch.zeros_like(xs)
    if dfinal is not None:
        dxs[:, L:] += dfinal.double()
    for k in range(W):
        dxs[:, k:k + L] += dy * w[:, k]
    dw = torch.stack([(dy * xs[:, k:k + L]).sum((0, 1)) for k in range(W)], 1)
    return {"dx": dxs[:, W - 1:], "dinit": dxs[:, :W - 1], "dweight": dw, "dbias": dy.sum((0, 1))}


def backward_rows(Bt, L, K, W, dtype):
    """Partial rows of a backward call, by its workspace (64 more where they are
    summed in two passes)."""
    from structured_state_space_ssd_amd._native import lib
    return lib.ssd_conv_backward_workspace_size(Bt, L, K, W, int(dtype == BF)) // (4 * K * (W + 1))


def check_exact_backward(ssd, Bt, L, K, W, dtype=F32, ends=True):
    x, w, b, init, dy, dfinal = integers(Bt, L, K, W, L + K, dtype)
    if not ends:
        init = dfinal = None
    got = ssd.conv_backward(x, w, b, dy, silu=False, init_state=init, dfinal_state=dfinal)
    want = exact_backward(x, w, dy, init, dfinal)
    for k in ("dweight", "dbias", "dx") + (("dinit",) if ends else ()):
        # (dx of at most 4 * 6 + 3 is exact in bf16 as well)
        assert torch.equal(got[k].double(), want[k]), (k, Bt, L, K, W)


# Rows around 2048, above which they are summed to 64 rows first: ceil(rows / 64) to
# each, so that 2049 rows of 33 leave the 63rd three and the 64th none, and 2112 none short.
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("rows", [1, 33, 2047, 2048, 2049, 2079, 2080, 2112, 2113, 3000])
def test_conv_backward_row_sums_exact(ssd, rows, W):
    K, tile = 5, 8
    two = 64 if rows > 2048 else 0
    for Bt, L in ((1, rows * tile), (1, rows * tile - 5), (rows, 3)):
        assert backward_rows(Bt, L, K, W, F32) == rows + two
        check_exact_backward(ssd, Bt, L, K, W)


def test_conv_backward_row_sums_see_every_row(ssd):
    """What the test above relies on: leaving any one tile's tokens out of the
    reference's sum changes every column of dbias."""
    x, w, b, init, dy, _ = integers(1, 2049 * 8 - 5, 5, 3, 1)
    whole = dy.double().sum((0, 1))
    tiles = torch.nn.functional.pad(dy[0].double(), (0, 0, 0, 5)).view(2049, 8, 5).sum(1)
    assert bool((whole - tiles != whole).all()) and torch.equal(tiles.sum(0), whole)
    assert torch.equal(ssd.conv_backward(x, w, b, dy, silu=False)["dbias"].double(), whole)


# A tile takes more than 8 tokens only where that leaves 131072 lanes: tiles of 16, 32,
# 64 and 128 tokens, the last one part full, with a ragged last vector of channels.
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("L,K,W,tile", [(1030, 8191, 4, 16), (1027, 8191, 2, 16), (2077, 8190, 3, 32),
                                        (4133, 8189, 4, 64), (4001, 16383, 4, 128)], ids=str)
def test_conv_backward_long_tiles_exact(ssd, L, K, W, tile, dtype):
    assert backward_rows(1, L, K, W, dtype) == -(-L // tile)
    check_exact_backward(ssd, 1, L, K, W, dtype, ends=tile != 64)


# Forward, a tile takes 16 tokens where that leaves 262144 lanes: two groups of 8 rows,
# over which the window, and in packed sequences the place, is carried.
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Bt,L,K,W", [(1, 2061, 8193, 4), (3, 687, 8190, 3), (2, 1039, 8191, 2)], ids=str)
def test_conv_forward_long_tiles_exact(ssd, Bt, L, K, W, dtype):
    assert Bt * -(-L // 16) * -(-K // 4) >= 262144
    x, w, b, init, _, _ = integers(Bt, L, K, W, L)
    x, init = x.to(dtype), init.to(dtype)
    for start in (init, None):
        y, final = ssd.conv_forward(x, w, b, silu=False, init_state=start, return_final_state=True)
        want, last = exact_forward(x, w, b, start)  # at most 4 * 6 + 3: exact in bf16 as well
        assert torch.equal(y.double(), want) and torch.equal(final.double(), last)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lengths", ["short", "mixed", "second_group"])
def test_conv_packed_long_tiles_exact(ssd, lengths, dtype):
    L, K, W = 2061, 8193, 4
    g = torch.Generator().manual_seed(3)
    if lengths == "second_group":  # every boundary in a tile's second group of 8 tokens
        cu = [0] + [16 * i + 9 + i % 7 for i in range(L // 16)] + [L]
    else:
        most = 6 if lengths == "short" else 60
        cu = [0]
        while cu[-1] < L:  # empty sequences among them
            cu.append(min(L, cu[-1] + int(torch.randint(0, most, (1,), generator=g))))
    x, w, b, _, _, _ = integers(1, L, K, W, 4)
    x = x.to(dtype)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, final = ssd.conv_forward(x, w, b, silu=False, cu_seqlens=c, return_final_state=True)
    want, last = exact_forward(x, w, b, None, cu)
    assert torch.equal(y.double(), want) and torch.equal(final.double(), last)


def test_conv_long_tiles_silu(ssd):
    """The activation on the longer tiles, forward and backward, under the bounds of
    the short ones (64-bit forms with all tokens at once)."""
    L, K, W = 2061, 8193, 4
    x, w, b, _, g = make(1, L, K, W, BF, 8)
    dy = torch.randn(1, L, K, generator=g).to(BF).cuda()
    y, got = ssd.conv_forward(x, w, b), ssd.conv_backward(x, w, b, dy)
    assert backward_rows(1, L, K, W, BF) == -(-L // 32)
    xs = torch.cat([x.new_zeros(1, W - 1, K), x], 1).double()
    terms = [w[:, k].double() * xs[:, k:k + L] for k in range(W)]
    v, mag = b.double() + sum(terms), b.double().abs() + sum(t.abs() for t in terms)
    want = R.silu(v)
    R.check("y", y, want.cpu(), (1.1 * (W + 1) * mag + want.abs() * (8 + 2 * v.abs())).cpu(), 1.0)
    gr, ga = dy.double() * R.silu_grad(v), dy.double().abs() * (1 + v.abs())
    dxs, ma = torch.zeros_like(xs), torch.zeros_like(xs)
    for k in range(W):
        dxs[:, k:k + L] += gr * w[:, k].double()
        ma[:, k:k + L] += ga * w[:, k].double().abs()
    ops = W + 14 + (W + 1) * float(mag.max())
    R.check("dx", got["dx"], dxs[:, W - 1:].cpu(), ma[:, W - 1:].cpu(), ops)
    # A column's sum: a tile's 32 tokens one after another, then at most 3 of its 65 rows
    # in each of 32 strands, then those
    R.check("dbias", got["dbias"], gr.sum((0, 1)).cpu(), ga.sum((0, 1)).cpu(), ops + 32 + 3 + 32)
    for k in range(W):
        R.check(("dweight", k), got["dweight"][:, k], (gr * xs[:, k:k + L]).sum((0, 1)).cpu(),
                (ga * xs[:, k:k + L].abs()).sum((0, 1)).cpu(), ops + 32 + 3 + 32)
