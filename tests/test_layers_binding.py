"""Refusals of the convolution and the normalisation, on the CPU: the binding's
own (shapes, types, layout, before any device check) and the C ABI's (every
call here fails its checks, so nothing is launched)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
f32, bf = torch.float32, torch.bfloat16
FAKE = ctypes.c_void_p(0x100000)


@pytest.fixture(scope="module")
def ssd():
    import structured_state_space_ssd_amd as m
    return m


@pytest.fixture(scope="module")
def lib(ssd):
    from structured_state_space_ssd_amd import _native
    return _native.lib


z = torch.zeros
CONV = dict(x=z(2, 6, 8, dtype=bf), weight=z(8, 4), bias=z(8))
CONV_BAD = [
    (ValueError, "x must be", dict(x=z(2, 8, dtype=bf))),
    (ValueError, "x must be", dict(weight=z(7, 4))),
    (ValueError, "weight is required", dict(weight=None)),
    (ValueError, "bias", dict(bias=z(9))),
    (TypeError, "bias", dict(bias=z(8, dtype=bf))),
    (TypeError, "weight", dict(weight=z(8, 4, dtype=bf))),
    (ValueError, "contiguous", dict(x=z(2, 8, 6, dtype=bf).transpose(1, 2))),
    (ValueError, "init_state", dict(init_state=z(2, 4, 8, dtype=bf))),
    (TypeError, "init_state", dict(init_state=z(2, 3, 8))),
    (ValueError, "split", dict(split=(4, 3))),
    (ValueError, "split", dict(split=(8, 0))),
    (ValueError, "split", dict(split=(2, 2, 2, 2))),
    (ValueError, "packed", dict(cu_seqlens=z(3, dtype=torch.int32))),
    (ValueError, "GPU", dict()),
]


@pytest.mark.parametrize("error,text,over", CONV_BAD, ids=[f"{t}-{i}" for i, (_, t, _) in enumerate(CONV_BAD)])
def test_conv_forward_refuses(ssd, error, text, over):
    with pytest.raises(error, match=text):
        ssd.conv_forward(**{**CONV, **over})


def test_conv_other_refusals(ssd, lib):
    x, w, b = CONV.values()
    with pytest.raises(ValueError, match="dy is required"):
        ssd.conv_backward(x, w, b, (z(2, 6, 4, dtype=bf), None))
    with pytest.raises(ValueError, match="split"):
        ssd.conv_backward(x, w, b, (z(2, 6, 4, dtype=bf), z(2, 6, 5, dtype=bf)))
    # too many workgroups
    one = _ptrs(0x100000)
    assert lib.ssd_conv_step(FAKE, FAKE, 1 << 20, FAKE, None, 1 << 20, 1 << 20, 4, 1, 1, None, 0, one, None) == -3


def test_conv_packed_refuses(ssd):
    a = dict(CONV, x=z(1, 6, 8, dtype=bf))
    with pytest.raises(ValueError, match="packed"):
        ssd.conv_forward(**a, cu_seqlens=z(2, dtype=torch.int32), init_state=z(1, 3, 8, dtype=bf))
    with pytest.raises(ValueError, match="cu_seqlens"):
        ssd.conv_forward(**a, cu_seqlens=z(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="cu_seqlens"):
        ssd.conv_forward(**a, cu_seqlens=z(2, dtype=torch.int64))


def test_conv_backward_and_step_refuse(ssd):
    with pytest.raises(ValueError, match="dy is required"):
        ssd.conv_backward(CONV["x"], CONV["weight"], None, None)
    with pytest.raises(ValueError, match="dy must have shape"):
        ssd.conv_backward(CONV["x"], CONV["weight"], None, z(2, 5, 8, dtype=bf))
    with pytest.raises(ValueError, match="split"):
        ssd.conv_backward(CONV["x"], CONV["weight"], None, (z(2, 6, 4, dtype=bf),))
    with pytest.raises(TypeError, match="dy"):
        ssd.conv_backward(CONV["x"], CONV["weight"], None, z(2, 6, 8))
    with pytest.raises(ValueError, match="dfinal_state"):
        ssd.conv_backward(CONV["x"], CONV["weight"], None, z(2, 6, 8, dtype=bf), dfinal_state=z(2, 2, 8, dtype=bf))
    with pytest.raises(ValueError, match="state"):
        ssd.conv_step(z(2, 4, 8, dtype=bf), z(2, 8, dtype=bf), z(8, 4))
    with pytest.raises(ValueError, match="state is required"):
        ssd.conv_step(None, z(2, 8, dtype=bf), z(8, 4))
    with pytest.raises(ValueError, match="GPU"):
        ssd.conv_step(z(2, 3, 8, dtype=bf), z(2, 8, dtype=bf), z(8, 4))


NORM_BAD = [
    (ValueError, "weight must have shape", dict(weight=z(9))),
    (TypeError, "weight", dict(weight=z(8, dtype=bf))),
    (ValueError, "exclude", dict(residual=z(4, 8), z=z(4, 8, dtype=bf))),
    (TypeError, "residual", dict(x=z(4, 8), residual=z(4, 8, dtype=bf))),
    (ValueError, "residual", dict(residual=z(8, 8)[::2])),
    (ValueError, "z must have shape", dict(z=z(5, 8, dtype=bf))),
    (ValueError, "contiguous", dict(x=z(8, 4, dtype=bf).t())),
    (ValueError, "evenly spaced", dict(x=z(4, 6, 8, dtype=bf)[:, :5])),
    (ValueError, "GPU", dict()),
]


@pytest.mark.parametrize("error,text,over", NORM_BAD, ids=[f"{t}-{i}" for i, (_, t, _) in enumerate(NORM_BAD)])
def test_norm_forward_refuses(ssd, error, text, over):
    with pytest.raises(error, match=text):
        ssd.norm_forward(**{**dict(x=z(4, 8, dtype=bf), weight=z(8), bias=z(8)), **over})


def test_norm_backward_refuses(ssd):
    a = dict(dy=z(4, 8, dtype=bf), x=z(4, 8), weight=z(8), mean=z(4), rstd=z(4))
    for error, text, over in ((ValueError, "rstd is required", dict(rstd=None)),
                              (ValueError, "mean must have shape", dict(mean=z(5))),
                              (TypeError, "x must be", dict(dy=z(4, 8), x=z(4, 8, dtype=bf))),
                              (TypeError, "dresidual", dict(dresidual=z(4, 8, dtype=bf))),
                              (ValueError, "exclude", dict(z=z(4, 8, dtype=bf), dresidual=z(4, 8))),
                              (TypeError, "with z", dict(z=z(4, 8, dtype=bf))),
                              (ValueError, "GPU", dict())):
        with pytest.raises(error, match=text):
            ssd.norm_backward(**{**a, **over})


def _ptrs(*addresses):
    return (ctypes.c_void_p * len(addresses))(*addresses)


def conv_c(lib, **kw):
    a = dict(x=FAKE, xb=48, xt=8, w=FAKE, b=None, init=None, cu=None, nseq=0, batch=2, seqlen=6,
             channels=8, width=4, silu=1, dtype=1, split=None, nsplit=0, y=_ptrs(0x100000), fin=None)
    a.update(kw)
    return lib.ssd_conv_forward(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(y=_ptrs(None)), -1),
    (dict(batch=0), -2), (dict(seqlen=0), -2), (dict(channels=0), -2), (dict(xt=-1), -2),
    (dict(seqlen=(1 << 30) + 1), -2),
    (dict(width=1), -3), (dict(width=5), -3), (dict(dtype=2), -3),
    (dict(split=(ctypes.c_int * 2)(4, 3), nsplit=2, y=_ptrs(1 << 20, 1 << 20)), -2),
    (dict(split=(ctypes.c_int * 2)(8, 0), nsplit=2, y=_ptrs(1 << 20, 1 << 20)), -2),
    (dict(split=(ctypes.c_int * 2)(1 << 30, 1 << 30), nsplit=2, y=_ptrs(1 << 20, 1 << 20)), -2),
    (dict(split=(ctypes.c_int * 2)(4, 4), nsplit=4, y=_ptrs(1 << 20, 1 << 20)), -2),
    (dict(split=(ctypes.c_int * 2)(4, 4), nsplit=2, y=_ptrs(1 << 20, None)), -1),
    (dict(cu=FAKE, nseq=2), -2), (dict(cu=FAKE, nseq=0, batch=1), -2),
    (dict(cu=FAKE, nseq=2, batch=1, init=FAKE), -3),
    (dict(batch=1 << 20, seqlen=1 << 30), -3),
])
def test_conv_c_abi_refuses(lib, kw, code):
    assert conv_c(lib, **kw) == code


def test_backward_workspaces(lib):
    n = lib.ssd_conv_backward_workspace_size(2, 6, 8, 4, 1)
    assert n > 0 and lib.ssd_conv_backward_workspace_size(2, 6, 8, 5, 1) == 0
    args = [FAKE, 48, 8, FAKE, None, None, None, 0, _ptrs(1 << 20), None, 2, 6, 8, 4, 1, 1, FAKE, FAKE,
            None, None]
    assert lib.ssd_conv_backward(*args, FAKE, n - 1, None) == -4
    assert lib.ssd_conv_backward(*args, None, n, None) == -4
    assert lib.ssd_conv_backward(*args, ctypes.c_void_p(0x100010), n, None) == -4
    m = lib.ssd_norm_backward_workspace_size(4, 8, 1, 1)
    assert m > 0 and lib.ssd_norm_backward_workspace_size(4, 16385, 1, 1) == 0
    assert lib.ssd_norm_backward_workspace_size(4, 8, 1, 0) * 2 == m
    args = [FAKE, FAKE, 8, 1, None, 0, FAKE, FAKE, FAKE, None, 4, 8, 1, FAKE, None, None, FAKE, FAKE]
    assert lib.ssd_norm_backward(*args, FAKE, m - 1, None) == -4
    args[4] = FAKE  # z without dz
    assert lib.ssd_norm_backward(*args, FAKE, m, None) == -1


def norm_c(lib, **kw):
    a = dict(x=FAKE, xs=8, res=None, rdt=0, z=None, zs=0, w=FAKE, b=None, rows=4, width=8, rms=0,
             eps=1e-5, dtype=1, y=FAKE, ro=None, mean=None, rstd=None)
    a.update(kw)
    return lib.ssd_norm_forward(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(res=FAKE), -1),
    (dict(rows=0), -2), (dict(width=0), -2), (dict(xs=-8), -2),
    (dict(width=16385), -3), (dict(dtype=3), -3), (dict(res=FAKE, ro=FAKE, z=FAKE), -3),
    (dict(res=FAKE, ro=FAKE, rdt=1, dtype=0), -3),
    (dict(eps=-1e-5), -6), (dict(eps=float("nan")), -6),
])
def test_norm_c_abi_refuses(lib, kw, code):
    assert norm_c(lib, **kw) == code


def scan_args(**over):
    a = dict(x=z(2, 6, 8, dtype=bf), dt=z(2, 6, 8, dtype=bf), A=z(8, 5), B=z(2, 6, 2, 5, dtype=bf),
             C=z(2, 6, 2, 5, dtype=bf), D=z(8))
    a.update(over)
    return a


SCAN_BAD = [
    (ValueError, "x must be", dict(A=z(8))),
    (ValueError, "x must be", dict(B=z(2, 6, 10, dtype=bf))),
    (ValueError, "x must be", dict(B=z(2, 5, 2, 5, dtype=bf))),
    (ValueError, "A must have shape", dict(A=z(9, 5))),
    (ValueError, "A must have shape", dict(A=z(8, 6))),
    (ValueError, "C must have shape", dict(C=z(2, 6, 1, 5, dtype=bf))),
    (ValueError, "dt must have shape", dict(dt=z(2, 6, 1, dtype=bf))),
    (TypeError, "dt must be", dict(dt=z(2, 6, 8))),
    (TypeError, "A must be", dict(A=z(8, 5, dtype=bf))),
    (ValueError, "groups", dict(B=z(2, 6, 3, 5, dtype=bf), C=z(2, 6, 3, 5, dtype=bf))),
    (ValueError, "groups must be contiguous", dict(B=z(2, 6, 2, 7, dtype=bf)[..., :5])),
    (ValueError, "last axis", dict(z=z(2, 8, 6, dtype=bf).transpose(1, 2))),
    (ValueError, "D must have shape", dict(D=z(7))),
    (ValueError, "dt_bias", dict(dt_bias=z(9))),
    (ValueError, "GPU", dict()),
]


@pytest.mark.parametrize("error,text,over", SCAN_BAD, ids=[f"{t}-{i}" for i, (_, t, _) in enumerate(SCAN_BAD)])
def test_selective_refuses(ssd, error, text, over):
    with pytest.raises(error, match=text):
        ssd.selective_forward(**scan_args(**over))
    with pytest.raises(error, match=text):
        ssd.selective_backward(**scan_args(**over), dy=z(2, 6, 8, dtype=bf))


def test_selective_more_refusals(ssd):
    with pytest.raises(ValueError, match="init_state"):
        ssd.selective_forward(**scan_args(init_state=z(2, 8, 4)))
    with pytest.raises(ValueError, match="dfinal_state"):
        ssd.selective_backward(**scan_args(dfinal_state=z(2, 4, 5)), dy=z(2, 6, 8, dtype=bf))
    with pytest.raises(ValueError, match="dy must have shape"):
        ssd.selective_backward(**scan_args(), dy=z(2, 6, 7, dtype=bf))
    one = {k: (v[:, 0] if k in ("x", "dt", "B", "C") else v) for k, v in scan_args().items()}
    with pytest.raises(ValueError, match="GPU"):
        ssd.selective_step(z(2, 8, 5), **one)
    with pytest.raises(ValueError, match="state must have shape"):
        ssd.selective_step(z(2, 8, 4), **one)
    with pytest.raises(ValueError, match="x must be"):
        ssd.selective_step(z(2, 8, 5), **dict(one, x=z(8, dtype=bf)))


def scan_c(lib, **kw):
    from structured_state_space_ssd_amd import _native
    strides, opts = kw.pop("strides", None), kw.pop("opts", None)
    a = dict(x=FAKE, dt=FAKE, A=FAKE, B=FAKE, C=FAKE, D=None, z=None, batch=2, seqlen=6, channels=8,
             ngroups=2, dstate=5, dtype=1, init=None, y=FAKE, fin=None, ws=None, bytes=0)
    a.update(kw)
    st = None if strides is None else ctypes.byref(_native.SsdSelectiveStrides(*strides))
    return lib.ssd_selective_forward(*a.values(), st, None if opts is None else ctypes.byref(opts), None)


def _opt(**kw):
    from structured_state_space_ssd_amd import _native
    return _native.SsdOptions(**kw)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(dt=None), -1), (dict(A=None), -1), (dict(B=None), -1), (dict(C=None), -1),
    (dict(y=None), -1), (dict(batch=0), -2), (dict(seqlen=0), -2), (dict(channels=0), -2),
    (dict(ngroups=0), -2), (dict(dstate=0), -2), (dict(ngroups=3), -2), (dict(seqlen=(1 << 30) + 1), -2),
    (dict(strides=(0, 0, 0, 0, 0, 0, 0, -1, 0, 0)), -2),
    (dict(dstate=65), -3), (dict(dtype=2), -3), (dict(batch=1 << 24), -3),
    # rows too long for offsets in 32 bits, whatever the inputs' strides
    (dict(channels=1 << 24, batch=1, strides=(0,) * 10), -3), (dict(strides=(0, 0, 0, 0, 0, 1 << 24, 0, 0, 0, 0)), -3),
    (dict(ws=FAKE, bytes=(2 * 2 * 32 + 32) * 64 - 1), -4), (dict(ws=ctypes.c_void_p(0x100010), bytes=1 << 30), -4),
    (dict(ws=None, bytes=1 << 30), -4),
], ids=str)
def test_selective_c_abi_refuses(lib, kw, code):
    assert scan_c(lib, **kw) == code


def test_selective_c_abi_options_and_workspaces(lib):
    assert scan_c(lib, opts=_opt(discretization=1)) == -6
    assert scan_c(lib, opts=_opt(dt_clamp=1, dt_min=1.0, dt_max=0.5)) == -6
    assert scan_c(lib, opts=_opt(dt_clamp=1, dt_min=float("nan"), dt_max=0.5)) == -6
    size = lib.ssd_selective_forward_workspace_size
    # B and C as float, the tokens rounded up to 32 and 32 to spare; segment states
    # where few channels have the token axis cut
    assert size(2, 6, 8, 2, 5, 1) == (2 * 2 * 32 + 32) * 2 * 8 * 4
    assert size(64, 4096, 5120, 1, 16, 1) == (64 * 4096 + 32) * 32 * 4
    assert size(1, 4096, 64, 1, 16, 1) > (4096 + 32) * 32 * 4 and size(1, 4096, 64, 1, 65, 1) == 0
    back = lib.ssd_selective_backward_workspace_size
    n = back(2, 6, 8, 2, 5, 1)
    assert n > 0
    args = [FAKE] * 5 + [None, None, None, FAKE, None, 2, 6, 8, 2, 5, 1] + [FAKE] * 5 + [None] * 4
    assert lib.ssd_selective_backward(*args, FAKE, n - 1, None, None, None) == -4
    args[8] = None
    assert lib.ssd_selective_backward(*args, FAKE, n, None, None, None) == -1
    args[8], args[6] = FAKE, FAKE  # z without dz
    assert lib.ssd_selective_backward(*args, FAKE, n, None, None, None) == -1
    # sizes whose products pass 32 bits
    assert back(8, 1 << 20, 8192, 1, 64, 0) > (1 << 32)


def test_norm_backward_wanted_refuses(ssd):
    a = dict(dy=z(4, 8, dtype=bf), x=z(4, 8, dtype=bf), weight=z(8), mean=None, rstd=z(4))
    with pytest.raises(ValueError, match="exclude"):
        ssd.norm_backward(**a, z=z(4, 8, dtype=bf), want_dresidual=True)
    for over in (dict(want_dbias=True), dict(want_dresidual=True), dict(z=z(4, 8, dtype=bf), want_dresidual=False)):
        with pytest.raises(ValueError, match="GPU"):
            ssd.norm_backward(**a, **over)


def test_selective_step_c_abi_token_strides(lib):
    """Only the strides between sequences are a single token's: the others may hold
    anything. (An invalid option is the last check, so nothing is launched.)"""
    from structured_state_space_ssd_amd import _native
    bad = _opt(discretization=1)
    args = [FAKE] * 6 + [None, None, 2, 8, 2, 5, 1, FAKE]
    for token in (8, -1, 1 << 40):
        st = _native.SsdSelectiveStrides(8, token, 8, token, 8, token, 10, token, 10, token)
        assert lib.ssd_selective_step(*args, ctypes.byref(st), ctypes.byref(bad), None) == -6
    st = _native.SsdSelectiveStrides(-8, 0, 8, 0, 8, 0, 10, 0, 10, 0)
    assert lib.ssd_selective_step(*args, ctypes.byref(st), ctypes.byref(bad), None) == -2


def test_grids_past_the_limit_refused_before_any_work(lib):
    """A grid takes fewer than 2^32 lanes. Every launch of a call is looked at
    before its first one: calls whose later kernels pass the limit are refused as
    unsupported, those just below it get to the workspace (missing here)."""
    def back(batch, seqlen, channels, ngroups, dstate):
        args = [FAKE] * 5 + [None, None, None, FAKE, None, batch, seqlen, channels, ngroups, dstate, 1]
        return lib.ssd_selective_backward(*args, *[FAKE] * 5, *[None] * 4, None, 0, None, None, None)

    # the sums of dB and dC: 4 tokens to a row of 1024 values at 64 states, 256 to a workgroup
    assert back(1, 1 << 24, 64, 1, 64) == -3 and back(1, (1 << 24) - 4, 64, 1, 64) == -4
    # 512 lanes to a workgroup at 32 states and more: 2^23 of them are too many
    assert back(1 << 20, 1, 512, 1, 32) == -3 and back((1 << 20) - 1, 1, 512, 1, 32) == -4
    # the sum of the rates' partial rows: 1024 lanes to 64 columns of channels x states
    assert back(1, 1, 1 << 23, 1, 32) == -3 and back(1, 1, (1 << 23) - 64, 1, 32) == -4
    assert back(1, 1, 1 << 22, 1, 64) == -3 and back(1, 1, 1 << 22, 1, 63) == -4

    def conv(batch, seqlen, channels, width):
        args = [FAKE, 0, 0, FAKE, None, None, None, 0, _ptrs(1 << 20), None, batch, seqlen, channels, width, 1, 1]
        return lib.ssd_conv_backward(*args, FAKE, FAKE, None, None, None, 0, None)

    # the sum of the filters' partial rows: channels x (width + 1) columns
    assert conv(1, 1, 1 << 26, 3) == -3 and conv(1, 1, (1 << 26) - 16, 3) == -4
    assert conv(1 << 20, 1 << 20, 64, 4) == -3  # the walk itself


def _far(*shape, dtype=f32):
    """A tensor of this shape that holds one element (its last axis one long or dense)."""
    return torch.zeros(1, dtype=dtype).expand(shape)


def test_sizes_past_an_int_refused(ssd):
    """The C ABI's sizes are ints; a size that one does not hold is refused, not cut to
    its low 32 bits (2^32 + 8 tokens would be 8)."""
    many = (1 << 32) + 8
    with pytest.raises(ValueError, match="2\\^31"):
        ssd.conv_forward(_far(1, many, 1), z(1, 4))
    with pytest.raises(ValueError, match="2\\^31"):
        ssd.conv_backward(_far(1, many, 1), z(1, 4), None, _far(1, many, 1))
    with pytest.raises(ValueError, match="2\\^31"):
        ssd.conv_step(_far(many, 3, 1), _far(many, 1), z(1, 4))
    with pytest.raises(ValueError, match="2\\^31"):
        ssd.conv_forward(z(1, 6, 8), z(8, 4), cu_seqlens=_far(many, dtype=torch.int32))
    scan = dict(x=_far(1, many, 1), dt=_far(1, many, 1), A=z(1, 1), B=_far(1, many, 1, 1), C=_far(1, many, 1, 1))
    for call in (ssd.selective_forward, lambda **a: ssd.selective_backward(**a, D=None, dy=scan["x"])):
        with pytest.raises(ValueError, match="2\\^31"):
            call(**scan)
    one = dict(x=_far(many, 1), dt=_far(many, 1), A=z(1, 1), B=_far(many, 1, 1), C=_far(many, 1, 1))
    with pytest.raises(ValueError, match="2\\^31"):
        ssd.selective_step(_far(many, 1, 1), **one)
    wide = _far(2, many)
    for call in (lambda: ssd.norm_forward(wide, _far(many)),
                 lambda: ssd.norm_backward(wide, wide, _far(many), None, z(2))):
        with pytest.raises(ValueError, match="2\\^31|contiguous"):
            call()


def test_selective_one_token_has_no_token_stride(lib):
    """A sequence of one token may come with any stride between tokens (torch leaves
    that of an axis of length one open): it is not looked at."""
    for token in (1 << 24, 1 << 40, -1):
        st = (8, token, 8, token, 8, token, 10, token, 10, token)
        assert scan_c(lib, seqlen=1, strides=st) == -4 and scan_c(lib, seqlen=2, strides=st) in (-2, -3)
