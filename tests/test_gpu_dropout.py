"""dropout_fwd / dropout_bwd (GPU): bit for bit against the draws in plain integers. A kept element is one fp32 product,
rounded once to the type, on both sides."""
import math

import pytest

torch = pytest.importorskip("torch")
import draws64 as D  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1), (1, 8), (3, 7), (5, 16), (2, 255), (7, 256), (9, 257), (33, 1001), (130, 2048), (4, 70000), (3000, 24), (1, 16384)]


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def draw(rows, cols, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * std).to(dtype)


def plain(x, p, seed, step, site):
    k = D.keep(*x.shape, p, seed, step, site).to(x.device)
    return torch.where(k, (x.float() * torch.tensor(D.factor(p), dtype=torch.float32)).to(x.dtype), torch.zeros_like(x))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(L, rows, cols, dtype):
    seed, step, site, p = -3 - (5 << 40), 7 + (9 << 32), 4000000000, 0.3
    x, dy = draw(rows, cols, dtype, 1), draw(rows, cols, dtype, 2)
    rng = L.dropout_rng(seed, step=step)
    y, ctx = L.dropout_fwd(x, p, rng, site=site)
    rng += 1  # the backward has its own copy
    assert torch.equal(y, plain(x, p, seed, step, site))
    assert torch.equal(L.dropout_bwd(dy, ctx), plain(dy, p, seed, step, site))
    z, _ = L.dropout_fwd(x, p, rng, site=site)
    assert torch.equal(z, plain(x, p, seed + 1, step + 1, site))


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 2.0 ** -16, 0.5, 1 - 2.0 ** -16, 1 - 2.0 ** -18, 1.0])
@pytest.mark.parametrize("cols", [1000, 1003])
def test_ends_of_p(L, p, cols):
    x = draw(70, cols, torch.float32, 1)
    rng = L.dropout_rng(5)
    y, ctx = L.dropout_fwd(x, p, rng)
    assert torch.equal(y, plain(x, p, 5, 0, 0)) and torch.equal(L.dropout_bwd(x, ctx), y)
    if p < 2.0 ** -17:
        assert torch.equal(y, x)
        assert torch.equal(L.dropout_fwd(x, p, None)[0], x)
    if p > 1 - 2.0 ** -17:
        assert (y == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,lead", [(96, 8), (96, 1), (33, 3), (260, 4)])
def test_strides_and_alignment_do_not_change_the_draws(L, cols, lead, dtype):
    x = draw(50, cols + 40, dtype, 1)
    out = torch.full_like(x, 7.0)
    rng = L.dropout_rng(11, step=2)
    y, _ = L.dropout_fwd(x[:, lead : lead + cols], 0.4, rng, y=out[:, lead : lead + cols])
    assert torch.equal(y, plain(x[:, lead : lead + cols], 0.4, 11, 2, 0))
    out[:, lead : lead + cols] = 7.0
    assert (out == 7.0).all()


@pytest.mark.parametrize("cols", [64, 65])
def test_what_is_dropped_is_zero_whatever_it_held(L, cols):
    x = torch.full((100, cols), math.nan, device="cuda")
    x[50:] = math.inf
    y, _ = L.dropout_fwd(x, 0.5, L.dropout_rng(1))
    k = D.keep(100, cols, 0.5, 1, 0, 0).cuda()
    assert (y[~k] == 0).all() and y[:50][k[:50]].isnan().all() and (y[50:][k[50:]] == math.inf).all()


def test_no_rows(L):
    x = torch.empty(0, 64, device="cuda")
    y, ctx = L.dropout_fwd(x, 0.5, L.dropout_rng(1))
    assert y.shape == x.shape and L.dropout_bwd(y, ctx).shape == x.shape


def test_graph_draws_anew_when_the_step_is_advanced(L):
    x = draw(200, 512, torch.bfloat16, 1)
    rng = L.dropout_rng(9)
    L.dropout_fwd(x, 0.2, rng)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, ctx = L.dropout_fwd(x, 0.2, rng, site=1)
        rng[1] += 1
        dx = L.dropout_bwd(x, ctx)
    for step in range(3):
        g.replay()
        want = plain(x, 0.2, 9, step, 1)
        assert torch.equal(y, want) and torch.equal(dx, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z, c = L.dropout_fwd(x, 0.2, rng, site=1, stream=s)
    d = L.dropout_bwd(x, c, stream=s)
    s.synchronize()
    assert torch.equal(z, plain(x, 0.2, 9, 3, 1)) and torch.equal(d, z)


@pytest.mark.parametrize("cols", [8192, 8191])
def test_offsets_past_32_bits(L, cols):
    rows = (1 << 32) // cols + 9
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    y, _ = L.dropout_fwd(x, 0.25, L.dropout_rng(3))
    for lo in (0, (1 << 31) // cols - 4, rows - 9):
        k = D.keep(9, cols, 0.25, 3, 0, 0, row0=lo).cuda()
        assert torch.equal(y[lo : lo + 9] != 0, k)
    assert abs(float((y != 0).sum(dtype=torch.float64)) / y.numel() - 0.75) < 5 * math.sqrt(0.1875 / y.numel())


def test_refusals(L):
    x = draw(4, 64, torch.bfloat16, 1)
    rng = L.dropout_rng(1)
    for p in (-0.1, 1.1, math.nan):
        with pytest.raises(ValueError, match="p is"):
            L.dropout_fwd(x, p, rng)
    with pytest.raises(ValueError, match="needs rng"):
        L.dropout_fwd(x, 0.1, None)
    with pytest.raises(ValueError, match="site"):
        L.dropout_fwd(x, 0.1, rng, site=-1)
    with pytest.raises(TypeError, match="rng"):
        L.dropout_fwd(x, 0.1, rng.int())
    with pytest.raises(TypeError, match="rng is not a CUDA tensor"):
        L.dropout_fwd(x, 0.1, rng.cpu())
    with pytest.raises(ValueError, match="rng has shape"):
        L.dropout_fwd(x, 0.1, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError, match="expected one of"):
        L.dropout_fwd(x.double(), 0.1, rng)
    with pytest.raises(ValueError, match="two dimensions"):
        L.dropout_fwd(x[0], 0.1, rng)
