"""Dropout on the GPU: the mask is the generator's to the bit, a kept value is off by its
scale's rounding, the product's and its type's."""
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


SIZES = [(1, 1), (5, 3), (1000, 8), (33, 9), (7, 255), (300, 333), (3, 5120), (1, 70001), (40000, 17)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_dropout(ssd, size, dtype):
    rows, D = size
    g = torch.Generator().manual_seed(rows + D)
    for p, pad, rng in ((0.1, 0, (0, 0)), (0.5, 3, ((1 << 64) - 5, (1 << 33) + 1)), (0.999, 8, (12345678901234, 1 << 63))):
        x = torch.randn(rows, D + pad, generator=g).to(dtype).cuda()[:, pad:]
        y = ssd.dropout(x, p, rng)
        want = B.dropped(x, p, rng)
        R.check((size, p), y, want, want.abs(), 3)
        state = torch.tensor([v - (1 << 64) if v >> 63 else v for v in rng], device="cuda")
        assert torch.equal(ssd.dropout(x, p, state), y)


def test_dropout_ends(ssd):
    x = torch.randn(3, 5, 40, device="cuda")
    x[0, 0, :3] = torch.tensor([float("nan"), float("inf"), float("-inf")])
    assert torch.equal(ssd.dropout(x, 0.0, None)[1:], x[1:]) and bool(ssd.dropout(x, 0.0, (1, 2))[0, 0, 0].isnan())
    assert bool((ssd.dropout(x, 1.0, (1, 2)) == 0).all())  # whatever was there
    # a share below half a step of 1/65536 drops nothing, one above drops some
    big = torch.ones(1000, 1000, device="cuda")
    assert bool((ssd.dropout(big, 0.49 / 65536, (1, 2)) == 1).all())
    assert int((ssd.dropout(big, 0.5 / 65536, (1, 2)) == 0).sum()) > 0
    # six standard deviations of a million draws
    for p in (0.1, 0.5):
        share = float((ssd.dropout(big, p, (3, 4)) == 0).double().mean())
        assert abs(share - p) < 6 * (p * (1 - p) / 1e6) ** 0.5
    # other seeds, offsets, rows and columns are other draws
    masks = [ssd.dropout(big, 0.5, rng) == 0 for rng in ((1, 0), (2, 0), (1, 1), (1 << 32, 0), (1, 1 << 32))]
    masks += [masks[0].roll(1, 0), masks[0].roll(1, 1), masks[0].roll(8, 1)]
    for i in range(len(masks)):
        for j in range(i):
            assert abs(float((masks[i] == masks[j]).double().mean()) - 0.5) < 6 * 0.5 / 1000


def test_dropout_captured(ssd):
    """A graph draws anew at every replay, from the state on the GPU; the mask of the
    backward is the forward's."""
    x, dy = torch.randn(100, 333, device="cuda").bfloat16(), torch.randn(100, 333, device="cuda").bfloat16()
    rng = torch.tensor([5, 0], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssd.dropout(x, 0.3, rng)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = ssd.dropout(x, 0.3, rng), ssd.dropout(dy, 0.3, rng)
    for k in range(4):
        rng[1] = k
        x.copy_(torch.randn(x.shape).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ssd.dropout(x, 0.3, (5, k))) and torch.equal(dx, ssd.dropout(dy, 0.3, (5, k)))
        assert bool(((y == 0) >= (dx == 0) & (x != 0)).all())


def test_dropout_large(ssd):
    """More than 2^32 elements; rows farther apart than that in bytes."""
    rows, D = 300000, 16384
    x = torch.ones(1, D, device="cuda", dtype=BF).expand(rows, D)
    y = ssd.dropout(x, 0.25, (1, 2))
    for k in (0, 1, 131071, 131072, 262144, rows - 1):
        assert torch.equal(y[k].cpu() != 0, B.kept(1, D, 0.25, 1, 2, first=k)[0]), k
    del y
    far = torch.empty((1 << 32) + 100, device="cuda", dtype=BF)
    x = far.as_strided((2, 100), (1 << 32, 1))
    x.copy_(torch.randn(2, 100))
    assert torch.equal(ssd.dropout(x, 0.25, (1, 2)), ssd.dropout(x.contiguous(), 0.25, (1, 2)))
