"""The plain 64-bit forms that the recurrent block's operators are tested against,
themselves against automatic differentiation, and the generator against its published
vectors (all on the CPU)."""
import numpy as np
import pytest

import block_refs as B
import layer_refs as R

torch = pytest.importorskip("torch")


def test_philox_known_answers():
    """The known-answer vectors that Philox 4x32-10's authors publish."""
    for counter, key, want in (
            ([0] * 4, (0, 0), [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
            ([0xffffffff] * 4, (0xffffffff,) * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
            ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], (0xa4093822, 0x299f31d0),
             [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])):
        assert B.philox(np.array(counter), key).tolist() == want


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 11], [2, 7, 9]], ids=str)
def test_recurrence_gradients(gated, cu):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    Bt, L, E = (2, 11, 5) if cu is None else (1, 11, 5)
    nseq = 0 if cu is None else len(cu) - 1
    leaves = dict(x=r(Bt, L, E), r=r(Bt, L, E) if gated else -r(Bt, L, E).abs(), i=r(Bt, L, E) if gated else None,
                  decay=r(E) if gated else None, z=r(Bt, L, E), init=r(Bt, E) if cu is None else None)
    dy, dfinal = r(Bt, L, E), r(nseq or Bt, E)
    got = B.recurrence(*leaves.values(), 8.0, cu, (dy, dfinal))
    t = {k: None if v is None else v.clone().requires_grad_() for k, v in leaves.items()}
    la = -8.0 * torch.nn.functional.softplus(t["decay"]) * torch.sigmoid(t["r"]) if gated else t["r"]
    a = torch.exp(la)
    u = torch.sqrt(1 - a * a) * torch.sigmoid(t["i"]) * t["x"] if gated else t["x"]
    spans = [(0, L)] if cu is None else list(zip(cu[:-1], cu[1:]))
    loss = 0
    for k, (p, q) in enumerate(spans):
        h = t["init"] if t["init"] is not None else torch.zeros(Bt, E, dtype=torch.float64)
        for n in range(p, q):
            h = a[:, n] * h + u[:, n]
            loss = loss + (dy[:, n] * h * torch.nn.functional.silu(t["z"][:, n])).sum()
        loss = loss + (dfinal[k] * h[0] if cu is not None else dfinal * h).sum()
    keys = [k for k, v in t.items() if v is not None]
    want = dict(zip(keys, torch.autograd.grad(loss, [t[k] for k in keys])))
    for k in keys:
        torch.testing.assert_close(got["d" + k], want[k], rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("pre,post", [(1, 1), (0, 1), (1, 0)])
def test_block_gradients(rms, pre, post):
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    rows, D, p, rng = 4, 9, 0.25, (3, 5)
    par = dict(x=r(rows, D), residual=r(rows, D), weight=r(D) if pre else None, bias=r(D) if pre else None,
               post_weight=r(D) if post else None, post_bias=r(D) if post else None, scale=r(D), z=r(rows, D))
    ref = B.Block(*par.values(), 1.5, -0.5, p, rng, 1e-5, rms)
    dy, dsum = r(rows, D) if pre else None, r(rows, D)
    got, _ = ref.grads(dy, dsum, ref.total)
    t = {k: None if v is None else v.clone().requires_grad_() for k, v in par.items()}

    def norm(v, w, b):
        v = v if rms else v - v.mean(-1, keepdim=True)
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w + b

    v = norm(t["x"], t["post_weight"], t["post_bias"]) if post else t["x"]
    v = v * t["scale"] * torch.nn.functional.silu(t["z"]) * B.kept(rows, D, p, *rng).double() / 0.75
    total = 1.5 * t["residual"] - 0.5 * v
    torch.testing.assert_close(ref.total, total.detach(), rtol=1e-12, atol=1e-12)
    loss = (total * dsum).sum()
    if pre:
        y = norm(total, t["weight"], t["bias"])
        torch.testing.assert_close(ref.y(ref.total)[0], y.detach(), rtol=1e-12, atol=1e-12)
        loss = loss + (y * dy).sum()
    keys = [k for k, v in t.items() if v is not None]
    for k, want in zip(keys, torch.autograd.grad(loss, [t[k] for k in keys])):
        torch.testing.assert_close(got["d" + k], want, rtol=1e-9, atol=1e-12)


def test_kept_share():
    """0.3 of 100000 elements within 6 standard deviations; nothing at 0, all at 1."""
    k = B.kept(100, 1000, 0.3, 7, 8)
    assert abs(float(k.double().mean()) - 0.7) < 6 * (0.21 / 100000) ** 0.5
    assert bool(B.kept(3, 20, 0.0, 1, 2).all()) and not bool(B.kept(3, 20, 1.0, 1, 2).any())
    assert R.U32 == 2.0 ** -24
