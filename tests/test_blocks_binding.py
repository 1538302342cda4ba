"""Refusals of the recurrence, the block norm and dropout, on the CPU: the binding's own
(shapes, types, layout, before any device check) and the C ABI's (every call here
fails its checks, so nothing is launched)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
f32, bf = torch.float32, torch.bfloat16
FAKE = ctypes.c_void_p(0x100000)
z = torch.zeros


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


@pytest.fixture(scope="module")
def lib(ssd):
    from structured_state_space_ssd_amd import _native
    return _native.lib


# ---- recurrence -------------------------------------------------------------------------

REC = dict(x=z(2, 6, 8, dtype=bf), r=z(2, 6, 8, dtype=bf), i=z(2, 6, 8, dtype=bf), decay=z(8))
REC_BAD = [
    (ValueError, "x is required", dict(x=None)),
    (ValueError, "r is required", dict(r=None)),
    (ValueError, "x must be", dict(x=z(2, 8, dtype=bf))),
    (ValueError, "go together", dict(i=None)),
    (ValueError, "go together", dict(decay=None)),
    (ValueError, "r must have shape", dict(r=z(2, 6, 7, dtype=bf))),
    (TypeError, "i must be", dict(i=z(2, 6, 8))),
    (ValueError, "decay must have shape", dict(decay=z(2, 8))),
    (TypeError, "decay must be", dict(decay=z(8, dtype=bf))),
    (ValueError, "last axis", dict(z=z(2, 8, 6, dtype=bf).transpose(1, 2))),
    (ValueError, "init_state", dict(init_state=z(2, 7))),
    (TypeError, "init_state", dict(init_state=z(2, 8, dtype=bf))),
    (ValueError, "packed", dict(cu_seqlens=z(3, dtype=torch.int32))),
    (ValueError, "GPU", dict()),
    (ValueError, "GPU", dict(i=None, decay=None)),
]


@pytest.mark.parametrize("error,text,over", REC_BAD, ids=[f"{t}-{i}" for i, (_, t, _) in enumerate(REC_BAD)])
def test_recurrence_refuses(ssd, error, text, over):
    a = {**REC, **over}
    with pytest.raises(error, match=text):
        ssd.recurrence_forward(**a)
    with pytest.raises(error, match=text):
        ssd.recurrence_backward(**a, dy=z(2, 6, 8, dtype=bf))


def test_recurrence_more_refusals(ssd):
    dy = z(2, 6, 8, dtype=bf)
    for error, text, over in ((ValueError, "dy is required", dict(dy=None)), (ValueError, "dy must", dict(dy=dy[:, :5])),
                              (ValueError, "dfinal_state", dict(dfinal_state=z(8))),
                              (ValueError, "states must have shape", dict(states=z(2, 2, 8))),
                              (TypeError, "states", dict(states=z(2, 1, 8, dtype=bf)))):
        with pytest.raises(error, match=text):
            ssd.recurrence_backward(**{**REC, "dy": dy, **over})
    one = {k: v[:, 0] if v.dim() == 3 else v for k, v in REC.items()}
    for error, text, state, over in ((ValueError, "state is required", None, {}), (ValueError, "state must", z(2, 9), {}),
                                     (TypeError, "state", z(2, 8, dtype=bf), {}), (ValueError, "x must be", z(2, 8), REC),
                                     (ValueError, "GPU", z(2, 8), {})):
        with pytest.raises(error, match=text):
            ssd.recurrence_step(state, **{**one, **over})
    packed = {k: v[:1] if v.dim() == 3 else v for k, v in REC.items()}
    with pytest.raises(ValueError, match="packed"):
        ssd.recurrence_forward(**packed, cu_seqlens=z(3, dtype=torch.int32), init_state=z(1, 8))
    with pytest.raises(ValueError, match="cu_seqlens"):
        ssd.recurrence_forward(**packed, cu_seqlens=z(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="cu_seqlens"):
        ssd.recurrence_forward(**packed, cu_seqlens=z(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="dfinal_state"):  # one for every sequence
        ssd.recurrence_backward(**packed, dy=dy[:1], cu_seqlens=z(3, dtype=torch.int32), dfinal_state=z(1, 8))


def _strides(*v):
    from structured_state_space_ssd_amd import _native
    return ctypes.byref(_native.SsdRecurrenceStrides(*v))


def rec_c(lib, **kw):
    st = kw.pop("strides", None)
    a = dict(x=FAKE, r=FAKE, i=FAKE, decay=FAKE, c=8.0, z=None, batch=2, seqlen=6, channels=8, dtype=1, init=None, cu=None,
             nseq=0, y=FAKE, fin=None, states=None, ws=None, bytes=0)
    a.update(kw)
    return lib.ssd_recurrence_forward(*a.values(), None if st is None else _strides(*st), None)


BAD_C = [
    (dict(x=None), -1), (dict(r=None), -1), (dict(y=None), -1), (dict(i=None), -1), (dict(decay=None), -3),
    (dict(batch=0), -2), (dict(seqlen=0), -2), (dict(channels=0), -2), (dict(batch=-1), -2),
    (dict(seqlen=(1 << 30) + 1), -2), (dict(dtype=2), -3), (dict(channels=1 << 24), -3),
    (dict(c=0.0), -6), (dict(c=-8.0), -6), (dict(c=float("nan")), -6), (dict(c=float("inf")), -6),
    (dict(strides=(48, 8, 48, 8, 48, -1, 48, 8)), -2), (dict(strides=(48, 8, -48, 8, 48, 8, 48, 8)), -2),
    (dict(strides=(48, 1 << 24, 48, 8, 48, 8, 48, 8)), -3),
    (dict(cu=FAKE, nseq=2), -2), (dict(cu=FAKE, nseq=0, batch=1), -2), (dict(cu=FAKE, nseq=(1 << 30) + 1, batch=1), -2),
    (dict(cu=FAKE, nseq=1 << 30, batch=1), -2),
    (dict(cu=FAKE, nseq=2, batch=1, init=FAKE), -3),
    (dict(batch=1 << 30, channels=1 << 20), -3),
    (dict(cu=FAKE, nseq=2, batch=1), -4), (dict(cu=FAKE, nseq=2, batch=1, ws=ctypes.c_void_p(0x100010), bytes=1 << 20), -4),
]


@pytest.mark.parametrize("kw,code", BAD_C, ids=[str(i) for i in range(len(BAD_C))])
def test_recurrence_c_abi_refuses(lib, kw, code):
    assert rec_c(lib, **kw) == code


def test_recurrence_c_abi_backward_and_step(lib):
    size = lib.ssd_recurrence_backward_workspace_size
    n = size(2, 6, 8, 0, 0, 1)
    assert n > 0 and size(2, 6, 8, 0, 0, 3) == 0 and size(2, 0, 8, 0, 0, 1) == 0
    # the states that the caller has not kept: one for every 16 tokens
    assert size(8, 64, 512, 0, 0, 1) - size(8, 64, 512, 0, 1, 1) == 8 * 4 * 512 * 4
    assert lib.ssd_recurrence_forward_workspace_size(1, 100, 8, 1, 1) - lib.ssd_recurrence_forward_workspace_size(
        1, 100, 8, 0, 1) == 512 + 256  # a code for each token, the rates

    def back(**kw):
        a = dict(x=FAKE, r=FAKE, i=FAKE, decay=FAKE, c=8.0, z=None, init=None, cu=None, nseq=0, states=None, dy=FAKE,
                 dfinal=None, batch=2, seqlen=6, channels=8, dtype=1, dx=FAKE, dr=FAKE, di=FAKE, ddecay=FAKE, dz=None,
                 dinit=None, ws=FAKE, bytes=n - 1)
        a.update(kw)
        return lib.ssd_recurrence_backward(*a.values(), None, None)

    assert back() == -4 and back(ws=None, bytes=n) == -4 and back(ws=ctypes.c_void_p(0x100010), bytes=n) == -4
    for kw in (dict(dy=None), dict(dx=None), dict(dr=None), dict(di=None), dict(ddecay=None), dict(z=FAKE), dict(i=None)):
        assert back(**kw) == -1
    assert back(decay=None) == -3 and back(cu=FAKE, nseq=2, batch=1, dinit=FAKE) == -3
    assert back(c=-1.0) == -6 and back(batch=0) == -2

    def step(strides=None, **kw):
        a = dict(state=FAKE, x=FAKE, r=FAKE, i=FAKE, decay=FAKE, c=-1.0, z=None, batch=2, channels=8, dtype=1, y=FAKE)
        a.update(kw)
        return lib.ssd_recurrence_step(*a.values(), None if strides is None else _strides(*strides), None)

    assert step() == -6 and step(state=None) == -1 and step(y=None) == -1 and step(batch=0) == -2 and step(dtype=5) == -3
    assert step(c=1.0, batch=1 << 30, channels=1 << 20) == -3
    # a single token's stride between tokens may be anything; between sequences it may not
    assert step((8, -1) * 4, c=1.0, batch=1 << 30, channels=1 << 20) == -3
    assert step((8, 1 << 40) * 4, c=1.0, batch=1 << 30, channels=1 << 20) == -3
    assert step((8, 0, -8, 0, 8, 0, 8, 0), c=1.0) == -2
    for token in (1 << 24, -1):  # the same for a sequence of one token
        assert rec_c(lib, seqlen=1, batch=1 << 30, channels=1 << 20, strides=(8, token) * 4) == -3


# ---- dropout ------------------------------------------------------------------------------

def test_dropout_refuses(ssd, lib):
    from structured_state_space_ssd_amd._native import SsdRandom
    x = z(4, 8, dtype=bf)
    for error, text, a in ((ValueError, "x is required", (None, 0.1, (1, 2))), (ValueError, "between 0 and 1", (x, 1.5, (1, 2))),
                           (ValueError, "between 0 and 1", (x, float("nan"), (1, 2))),
                           (ValueError, "between 0 and 1", (x, -0.1, (1, 2))), (ValueError, "rng is required", (x, 0.1, None)),
                           (TypeError, "integers", (x, 0.1, (1.5, 2))), (ValueError, "rng must have shape", (x, 0.1, z(3, dtype=torch.int64))),
                           (TypeError, "rng must be", (x, 0.1, z(2))), (ValueError, "evenly spaced", (z(4, 6, 8)[:, ::2][:, :, :4][:2, :2], 0.1, (1, 2))),
                           (ValueError, "last axis", (x.t(), 0.1, (1, 2))), (ValueError, "GPU", (x, 0.1, (1, 2))),
                           (ValueError, "GPU", (x, 0, None))):
        if text == "evenly spaced":
            a = (z(4, 6, 8)[:3, :5, :4], 0.1, (1, 2))
        with pytest.raises(error, match=text):
            ssd.dropout(*a)

    def c(p=0.5, state=None, rows=4, width=8, dtype=1, x=FAKE, y=FAKE, stride=8):
        return lib.ssd_dropout(x, stride, rows, width, ctypes.byref(SsdRandom(p, 1, 2, state)), dtype, y, None)

    assert c(x=None) == -1 and c(y=None) == -1 and lib.ssd_dropout(FAKE, 8, 4, 8, None, 1, FAKE, None) == -1
    assert c(rows=0) == -2 and c(width=0) == -2 and c(stride=-8) == -2
    assert c(dtype=2) == -3 and c(rows=1 << 31) == -3 and c(width=(1 << 30) + 1) == -3 and c(state=0x100004) == -3
    assert c(p=-0.1) == -6 and c(p=1.1) == -6 and c(p=float("nan")) == -6


# ---- block norm -----------------------------------------------------------------------------

BLOCK = dict(x=z(4, 8, dtype=bf), residual=z(4, 8), weight=z(8), bias=z(8), post_weight=z(8), post_bias=z(8), scale=z(8),
             z=z(4, 8, dtype=bf))
BLOCK_BAD = [
    (ValueError, "x is required", dict(x=None)),
    (ValueError, "residual is required", dict(residual=None)),
    (ValueError, "residual must have shape", dict(residual=z(4, 7))),
    (TypeError, "residual must be float32 or", dict(residual=z(4, 8, dtype=torch.float16))),
    (ValueError, "weight or post_weight", dict(weight=None, bias=None, post_weight=None, post_bias=None)),
    (ValueError, "bias without its weight", dict(weight=None)),
    (ValueError, "post_bias without its weight", dict(post_weight=None)),
    (ValueError, "weight must have shape", dict(weight=z(7))),
    (TypeError, "post_bias must be", dict(post_bias=z(8, dtype=bf))),
    (ValueError, "scale must have shape", dict(scale=z(4, 8))),
    (ValueError, "z must have shape", dict(z=z(8, dtype=bf))),
    (TypeError, "z must be", dict(z=z(4, 8))),
    (ValueError, "rng is required", dict(p=0.1)),
    (ValueError, "between 0 and 1", dict(p=2, rng=(1, 2))),
    (ValueError, "evenly spaced", dict(x=z(4, 6, 8, dtype=bf)[:3, :5], residual=z(3, 5, 8), z=None)),
    (ValueError, "GPU", dict()),
]


@pytest.mark.parametrize("error,text,over", BLOCK_BAD, ids=[f"{t}-{i}" for i, (_, t, _) in enumerate(BLOCK_BAD)])
def test_block_norm_refuses(ssd, error, text, over):
    with pytest.raises(error, match=text):
        ssd.block_norm_forward(**{**BLOCK, **over})


def test_block_norm_backward_refuses(ssd):
    a = {k: v for k, v in BLOCK.items() if k != "residual"}
    a.update(dy=z(4, 8, dtype=bf), dsum=z(4, 8), total=z(4, 8), stats=(z(4), z(4), z(4), z(4)))
    for error, text, over in (
            (ValueError, "stats is required", dict(stats=None)), (ValueError, "total is required", dict(total=None)),
            (ValueError, "dy goes with weight", dict(dy=None)),
            (ValueError, "dy goes with weight", dict(weight=None, bias=None)),
            (ValueError, "dy must have shape", dict(dy=z(4, 7, dtype=bf))), (TypeError, "dsum must be", dict(dsum=z(4, 8, dtype=bf))),
            (TypeError, "total must be float32 or", dict(total=z(4, 8, dtype=torch.float16))),
            (ValueError, "rstd is required", dict(stats=(z(4), None, z(4), z(4)))),
            (ValueError, "post_rstd is required", dict(stats=(z(4), z(4), z(4), None))),
            (ValueError, "mean must have shape", dict(stats=(z(3), z(4), z(4), z(4)))),
            (ValueError, "GPU", dict()), (ValueError, "GPU", dict(stats=(None, z(4), None, z(4)), dsum=None))):
        with pytest.raises(error, match=text):
            ssd.block_norm_backward(**{**a, **over})


def block_c(lib, **kw):
    from structured_state_space_ssd_amd._native import SsdBlock, SsdRandom
    o = dict(w=0x100000, b=None, pw=0x100000, pb=None, s=None, alpha=1.0, beta=1.0, rms=0, eps=1e-5)
    o.update({k: kw.pop(k) for k in list(kw) if k in o})
    p = kw.pop("p", None)
    a = dict(x=FAKE, xs=8, res=FAKE, rdt=0, z=None, zs=0, block=ctypes.byref(SsdBlock(*o.values())),
             random=None if p is None else ctypes.byref(SsdRandom(p, 1, 2, None)), rows=4, width=8, dtype=1, y=FAKE, sum=FAKE,
             mean=None, rstd=None, pm=None, pr=None)
    a.update(kw)
    return lib.ssd_block_norm_forward(*a.values(), None)


BLOCK_C = [
    (dict(x=None), -1), (dict(res=None), -1), (dict(sum=None), -1), (dict(y=None), -1), (dict(block=None), -1),
    (dict(w=None, pw=None), -1), (dict(w=None, b=0x100000), -1), (dict(pw=None, pb=0x100000), -1),
    (dict(rows=0), -2), (dict(width=0), -2), (dict(xs=-8), -2), (dict(z=FAKE, zs=-8), -2),
    (dict(width=8193), -3), (dict(rows=1 << 31), -3), (dict(dtype=2), -3), (dict(rdt=1, dtype=0), -3), (dict(rdt=2), -3),
    (dict(alpha=float("inf")), -6), (dict(beta=float("nan")), -6), (dict(eps=-1.0), -6), (dict(eps=float("nan")), -6),
    (dict(p=1.5), -6),
]


@pytest.mark.parametrize("kw,code", BLOCK_C, ids=[str(i) for i in range(len(BLOCK_C))])
def test_block_norm_c_abi_refuses(lib, kw, code):
    assert block_c(lib, **kw) == code


def test_block_norm_c_abi_backward(lib):
    from structured_state_space_ssd_amd._native import SsdBlock
    size = lib.ssd_block_norm_backward_workspace_size
    n = size(4, 8, 1)
    assert n > 0 and size(4, 8193, 1) == 0 and size(0, 8, 1) == 0 and size(4, 8, 2) == 0 and size(1 << 31, 8, 1) == 0

    def c(w=0x100000, pw=0x100000, s=0x100000, rms=0, **kw):
        a = dict(dy=FAKE, dsum=None, x=FAKE, xs=8, sum=FAKE, sdt=0, z=None, zs=0,
                 block=ctypes.byref(SsdBlock(w, None, pw, None, s, 1.0, 1.0, rms, 0.0)), random=None, mean=FAKE, rstd=FAKE,
                 pm=FAKE, pr=FAKE, rows=4, width=8, dtype=1, dx=FAKE, dres=FAKE, dz=None, dw=FAKE, db=FAKE, dpw=FAKE,
                 dpb=FAKE, ds=FAKE, ws=FAKE, bytes=n - 1)
        a.update(kw)
        return lib.ssd_block_norm_backward(*a.values(), None)

    assert c() == -4 and c(ws=None, bytes=n) == -4
    for kw in (dict(dy=None), dict(sum=None), dict(rstd=None), dict(mean=None), dict(pm=None), dict(pr=None), dict(dx=None),
               dict(dres=None), dict(x=None), dict(z=FAKE)):
        assert c(**kw) == -1, kw
    assert c(rms=1, mean=None, pm=None) == -4
    # gradients of what is not there
    for kw in (dict(w=None), dict(w=None, dy=None, db=None), dict(pw=None), dict(pw=None, dpw=None), dict(s=None)):
        assert c(**kw) == -3, kw


def test_sizes_past_an_int_refused(ssd):
    far = lambda *shape, dtype=f32: torch.zeros(1, dtype=dtype).expand(shape)  # noqa: E731
    many = (1 << 32) + 8
    with pytest.raises(ValueError, match="2\\^31"):
        ssd.recurrence_forward(far(1, many, 1), far(1, many, 1))
    with pytest.raises(ValueError, match="2\\^31"):
        ssd.recurrence_backward(far(1, many, 1), far(1, many, 1), None, None, far(1, many, 1))
    with pytest.raises(ValueError, match="2\\^31"):
        ssd.recurrence_step(far(many, 1), far(many, 1), far(many, 1))
    with pytest.raises(ValueError, match="2\\^31|contiguous"):
        ssd.dropout(far(2, many), 0.5, (1, 2))
    with pytest.raises(ValueError, match="2\\^31|contiguous"):
        ssd.block_norm_forward(far(2, many), far(2, many), far(many))
