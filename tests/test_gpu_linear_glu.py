"""linear_glu_fwd / linear_glu_bwd (GPU): products of small whole numbers bit for bit, and everything else against the
formulas in 64 bits. Products of 16-bit values are exact in fp32; an accumulation step of 16 of them keeps at least 22 bits
of the largest term, so K / 16 + 8 steps of 2^-22 of the sum of magnitudes bound a sum over K however it is cut."""
import math

import pytest

torch = pytest.importorskip("torch")
import plain64 as P  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
ACTS = ["silu", "gelu", "relu", "none"]
# tokens, in, out: single tokens, the borders of the few-token forms and of the tiles, ragged and long ones
SHAPES = [(1, 64, 64), (1, 2048, 1024), (2, 520, 72), (4, 1024, 24), (5, 64, 8), (7, 72, 200), (16, 512, 136), (17, 256, 8), (33, 8, 256), (64, 640, 320),
          (65, 128, 128), (129, 200, 264), (255, 4096, 520), (300, 1032, 520), (513, 768, 768), (2048, 264, 1024), (700, 2048, 2056), (2600, 2568, 1288)]


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def draw(rows, cols, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * std + mean).to(dtype)


def whole(rows, cols, dtype, seed, most=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device="cuda").to(dtype)


def sum_error(K):
    return (K / 16 + 8) * 2.0 ** -22


def logistic_error(z, act):
    """Relative error bound of s(u): ex2.approx and rcp.approx (2 ulp each) and four roundings of u."""
    if act in ("none", "relu"):
        return torch.zeros_like(z)
    u = 1.6 * (z.abs() + 0.045 * z.abs() ** 3) if act == "gelu" else z.abs()
    return (16 + 4 * u.clamp(max=90)) * P.U


def slope_error(z, act):
    if act in ("none", "relu"):
        return torch.zeros_like(z)
    w = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3) if act == "gelu" else z
    du = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z) if act == "gelu" else torch.ones_like(z)
    s = torch.sigmoid(w)
    return 2 * logistic_error(z, act) * (s + z.abs() * s * torch.sigmoid(-w) * du) + z.abs() * du * s * P.U


def check_fwd(y, h, x, w, b, act):
    """y: the two factors' errors times the other factor; no slope here passes 1.13."""
    dt, K, N = x.dtype, x.shape[1], w.shape[0] // 2
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if b is not None:
        z, mag = z + b.double(), mag + b.double().abs()
    dz = sum_error(K) * mag + P.U * z.abs()
    if h is not None:
        P.assert_within(h, z, dz + P.half(dt) * (z.abs() + dz) + P.tiny(dt), "h")
    zg, zu, dg, du = z[:, :N], z[:, N:], dz[:, :N], dz[:, N:]
    a = P.act(zg, act)
    da = 1.2 * dg + logistic_error(zg, act) * a.abs() + 1e-35
    want = a * zu
    tol = da * (zu.abs() + du) + a.abs() * du + P.U * want.abs()
    P.assert_within(y, want, tol + P.half(dt) * (want.abs() + tol) + P.tiny(dt), "y")


def check_bwd(g, dy, x, w, h, act):
    dt, (M, N), K = dy.dtype, dy.shape, w.shape[1]
    d, zg, zu = dy.double(), h[:, :N].double(), h[:, N:].double()
    a, s = P.act(zg, act), P.slope(zg, act)
    dz = torch.cat((d * zu * s, d * a), 1)
    e32 = torch.cat(((d * zu).abs() * slope_error(zg, act), (d * a).abs() * logistic_error(zg, act)), 1) + 3 * P.U * dz.abs() + 1e-37
    e16 = e32 + P.half(dt) * (dz.abs() + e32) + P.tiny(dt)
    if g.dbias is not None:  # rows of a thread, its row lanes, the row blocks' partial sums and their lanes
        n = M / 64 + 48
        P.assert_within(g.dbias, dz.sum(0), n * P.U * dz.abs().sum(0) + e32.sum(0), "dbias")
    if g.dx is not None:
        wd = w.double()
        want, mag = dz @ wd, (dz.abs() + e16) @ wd.abs()
        tol = e16 @ wd.abs() + sum_error(2 * N) * mag
        P.assert_within(g.dx, want, tol + P.half(dt) * (want.abs() + tol) + P.tiny(dt), "dx")
    if g.dw is not None:
        xd = x.double()
        want, mag = dz.t() @ xd, (dz.abs() + e16).t() @ xd.abs()
        tol = e16.t() @ xd.abs() + sum_error(M) * mag
        P.assert_within(g.dw, want, tol + P.half(dt) * (want.abs() + tol) + P.tiny(dt), "dw")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_whole_number_products_are_exact(L, M, K, N, dtype):
    """Entries up to 2, no activation: z up to 4 K + 2 and sums below 2^24 are exact in fp32, their product below 2^24 too up
    to K = 1000 (2 deviations of a sum are 4 sqrt(K)), and y is rounded once. A gate and an up column that
    were mixed up, or a token out of place, would show."""
    x, w, b, dy = whole(M, K, dtype, 1), whole(2 * N, K, dtype, 2), whole(1, 2 * N, dtype, 3)[0], whole(M, N, dtype, 4)
    y, ctx = L.linear_glu_fwd(x, w, b, act="none", save="h")
    z = x.double() @ w.double().t() + b.double()
    assert torch.equal(ctx.h, z.to(dtype))
    assert torch.equal(y, (z[:, :N] * z[:, N:]).to(torch.float32).to(dtype))
    y2, ctx2 = L.linear_glu_fwd(x, w, b, act="none")
    assert torch.equal(y, y2) and ctx2.h is None
    ctx.h = whole(M, 2 * N, dtype, 5)
    g = L.linear_glu_bwd(dy, x, w, ctx)
    dz = torch.cat((dy.double() * ctx.h[:, N:].double(), dy.double() * ctx.h[:, :N].double()), 1)
    assert torch.equal(g.dx, (dz @ w.double()).to(dtype))
    assert torch.equal(g.dw, (dz.t() @ x.double()).to(dtype))
    assert torch.equal(g.dbias, dz.sum(0).float())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act,bias", [("silu", False), ("gelu", True), ("relu", True), ("none", False)])
def test_forward_and_backward(L, M, K, N, dtype, act, bias):
    x, w = draw(M, K, dtype, 1), draw(2 * N, K, dtype, 2, 1.5 / math.sqrt(K))
    b = draw(1, 2 * N, dtype, 3, 0.1)[0] if bias else None
    y, ctx = L.linear_glu_fwd(x, w, b, act=act, save="h")
    check_fwd(y, ctx.h, x, w, b, act)
    y2, _ = L.linear_glu_fwd(x, w, b, act=act)
    assert torch.equal(y, y2)
    dy = draw(M, N, dtype, 4, 0.1)
    g = L.linear_glu_bwd(dy, x, w, ctx, dbias=bias)
    assert (g.dbias is not None) == bias
    check_bwd(g, dy, x, w, ctx.h, act)
    again = L.linear_glu_bwd(dy, x, w, ctx, dbias=bias)
    assert torch.equal(g.dx, again.dx) and torch.equal(g.dw, again.dw) and (not bias or torch.equal(g.dbias, again.dbias))
    L.sync_status()


@pytest.mark.parametrize("M", [1, 3, 40, 100, 400])
@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_given_buffers(L, M, dtype):
    """Rows with strides of their own; what lies between and behind them stays as it was."""
    K, N = 136, 72
    x, w, dy = draw(M, K + 24, dtype, 1)[:, 8 : 8 + K], draw(2 * N, K, dtype, 2, 0.1), draw(M, N + 8, dtype, 3)[:, :N]
    out, dxo = torch.full((M + 2, N + 16), 7.0, dtype=dtype, device="cuda"), torch.full((M + 2, K + 40), 7.0, dtype=dtype, device="cuda")
    ctx = L.LinearGluCtx(h=torch.empty(M, 2 * N, dtype=dtype, device="cuda"))
    h = ctx.h
    y, ctx = L.linear_glu_fwd(x, w, save="h", y=out[:M, 8 : 8 + N], ctx=ctx)
    assert ctx.h is h and y.data_ptr() == out[:, 8:].data_ptr()
    check_fwd(y, h, x, w, None, "silu")
    g = L.linear_glu_grads(M, K, N, dtype=dtype)
    g.dx = dxo[:M, 16 : 16 + K]
    L.linear_glu_bwd(dy, x, w, ctx, grads=g)
    check_bwd(g, dy, x, w, h, "silu")
    for t, lo, n in ((out, 8, N), (dxo, 16, K)):
        t[:M, lo : lo + n] = 7.0
        assert (t == 7.0).all()


@pytest.mark.parametrize("parts", [("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ("dw", "dbias")])
def test_only_the_gradients_asked_for(L, parts):
    M, K, N = 150, 128, 192
    x, w, dy = draw(M, K, torch.bfloat16, 1), draw(2 * N, K, torch.bfloat16, 2, 0.1), draw(M, N, torch.bfloat16, 3)
    _, ctx = L.linear_glu_fwd(x, w, save="h")
    g = L.linear_glu_grads(M, K, N, dx="dx" in parts, dw="dw" in parts, bias="dbias" in parts)
    L.linear_glu_bwd(dy, x if "dw" in parts else None, w, ctx, grads=g)
    check_bwd(g, dy, x, w, ctx.h, "silu")
    full = L.linear_glu_bwd(dy, x, w, ctx)
    for k in parts:
        assert torch.equal(getattr(g, k), getattr(full, k)), k


def test_no_tokens(L):
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), draw(64, 64, torch.bfloat16, 1)
    y, ctx = L.linear_glu_fwd(x, w, save="h")
    assert y.shape == (0, 32)
    g = L.linear_glu_bwd(y, x, w, ctx)
    assert g.dx.shape == (0, 64) and (g.dw == 0).all() and (g.dbias == 0).all()


@pytest.mark.parametrize("M", [1, 3, 50, 130, 700])
@pytest.mark.parametrize("act", ACTS)
def test_infinities_and_nan_stay_where_they_are(L, M, act):
    """A NaN of a token reaches that token's outputs alone; one of a weight row its own output alone. Large finite values
    saturate as the formula does."""
    K, N = 64, 96
    x, w = draw(M, K, torch.bfloat16, 1), draw(2 * N, K, torch.bfloat16, 2, 0.2)
    w[5, 3] = math.nan
    w[N + 40, 2] = math.inf
    clean = torch.ones(N, dtype=torch.bool, device="cuda")
    clean[5] = clean[40] = False
    if M > 2:
        x[1, 0] = math.nan
    y, ctx = L.linear_glu_fwd(x, w, act=act, save="h")
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    if M > 2:
        assert y[1].isnan().all()
        rows[1] = False
    assert y[rows][:, 5].isnan().all() and not y[rows][:, 40].isfinite().any()
    assert y[rows][:, clean].isfinite().all()
    dy = draw(M, N, torch.bfloat16, 3)
    h = draw(M, 2 * N, torch.bfloat16, 4)
    h[0, 7], h[0, N + 9] = math.nan, math.nan
    g = L.linear_glu_bwd(dy, x.nan_to_num(), w.nan_to_num(0, 0, 0), L.LinearGluCtx(act=act, h=h))
    assert g.dx[0].isnan().all() and g.dx[1:].isfinite().all()
    bad = {N + 7, 9} if act == "none" else {7, N + 7, 9}  # without an activation the gate's own gradient does not read it
    assert {int(i) for i in g.dw.isnan().any(1).nonzero().flatten()} == bad
    assert {int(i) for i in g.dbias.isnan().nonzero().flatten()} == bad


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_pre_activations(L, act):
    """Gates of bf16's whole range: the activation is z or 0 far out and its slope 1 or 0, never NaN."""
    N = 64
    z = torch.logspace(-3, 38, N, device="cuda", dtype=torch.float64)
    z = torch.stack((z, -z)).to(torch.bfloat16)
    h = torch.cat((z, torch.ones_like(z)), 1)
    dy, w, x = torch.ones(2, N, dtype=torch.bfloat16, device="cuda"), torch.eye(2 * N, dtype=torch.bfloat16, device="cuda"), torch.ones(2, 2 * N, dtype=torch.bfloat16, device="cuda")
    g = L.linear_glu_bwd(dy, x, w, L.LinearGluCtx(act=act, h=h))
    want = torch.cat((P.slope(z.double(), act).nan_to_num(0.0), P.act(z.double(), act)), 1)
    far = z.double().abs() > 1e4
    want[:, :N] = torch.where(far, (z > 0).double(), want[:, :N])
    want[:, N:] = torch.where(far, z.double().clamp_min(0), want[:, N:])
    # beyond 5 the slope's factor s (1 - s) has vanished beside its own rounding, and the logistic function's (16 + 4 * 90) 2^-24
    # stays below a fortieth of the output's half step
    tol = torch.cat((slope_error(z.double().clamp(-5, 5), act), logistic_error(z.double().clamp(-5, 5), act) * want[:, N:].abs()), 1) + 1e-35
    P.assert_within(g.dx, want, tol + P.half(torch.bfloat16) * (want.abs() + tol) * 1.03 + P.tiny(torch.bfloat16), "dx")


def test_gradients_agree_with_differences(L):
    """The loss sum(c y) along a direction of w: with fp16 tensors and steps of 2^-4 the difference of two forwards holds the
    slope to the outputs' roundings, sqrt(M N) of them at random, and the third-order term of the step."""
    M, K, N = 64, 64, 96
    dt = torch.float16
    x, w, c = draw(M, K, dt, 1), draw(2 * N, K, dt, 2, 0.1), draw(M, N, dt, 3)
    step = 2.0 ** -4
    y, ctx = L.linear_glu_fwd(x, w, save="h")
    g = L.linear_glu_bwd(c, x, w, ctx)
    v = (g.dw.float() / g.dw.float().abs().mean() * 0.1).clamp(-0.3, 0.3)  # uphill, so that the slope is large
    up, down = (w.double() + s * step * v.double() for s in (1, -1))
    f = [(L.linear_glu_fwd(x, t.to(dt), save="none")[0].double() * c.double()).sum() for t in (up, down)]
    moved = [t.to(dt).double() for t in (up, down)]
    slope = (g.dw.double() * (moved[0] - moved[1])).sum()
    # the same difference of the formula in 64 bits says what the step itself costs
    def loss(t):
        z = x.double() @ t.t()
        return (P.act(z[:, :N], "silu") * z[:, N:] * c.double()).sum()
    cost = (loss(moved[0]) - loss(moved[1]) - (f[0] - f[1])).abs()
    noise = P.half(dt) * float((y.double() * c.double()).norm()) * 6  # two sums of independent roundings, six deviations
    assert float(cost) < noise
    curve = ((loss(moved[0]) - loss(moved[1])) - slope).abs()
    t64 = w.double().requires_grad_(True)
    exact = torch.autograd.grad(loss(t64), t64)[0]
    assert float((slope - (exact * (moved[0] - moved[1])).sum()).abs()) < 6 * P.half(dt) * float((g.dw.double() * (moved[0] - moved[1])).norm()) * 3 + 1e-3 * float(slope.abs())
    assert float(curve) < 0.1 * float(slope.abs()) + noise


@pytest.mark.parametrize("M", [1, 60, 500])
def test_other_stream_and_graph(L, M):
    """On a stream of its own, and captured and replayed on new contents; two captured graphs with a workspace each."""
    K, N, dt = 192, 160, torch.bfloat16
    x, w, dy = draw(M, K, dt, 1), draw(2 * N, K, dt, 2, 0.1), draw(M, N, dt, 3)
    y0, c0 = L.linear_glu_fwd(x, w, save="h")
    g0 = L.linear_glu_bwd(dy, x, w, c0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y1, c1 = L.linear_glu_fwd(x, w, save="h", stream=s)
    g1 = L.linear_glu_bwd(dy, x, w, c1, stream=s)
    s.synchronize()
    for a, b in ((y0, y1), (g0.dx, g1.dx), (g0.dw, g1.dw), (g0.dbias, g1.dbias)):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y, c = L.linear_glu_fwd(x, w, save="h")
            g = L.linear_glu_bwd(dy, x, w, c)
        graphs.append((gr, y, g))
    x.copy_(draw(M, K, dt, 11))
    y0, c0 = L.linear_glu_fwd(x, w, save="h")
    g0 = L.linear_glu_bwd(dy, x, w, c0)
    for gr, y, g in graphs + graphs:
        gr.replay()
        for a, b in ((y0, y), (g0.dx, g.dx), (g0.dw, g.dw), (g0.dbias, g.dbias)):
            assert torch.equal(a, b)
    L.sync_status()


def test_offsets_past_32_bits(L):
    """More than 2^32 bytes of z and of dz; rows from both ends against the same rows alone."""
    M, K, N, dt = 70000, 64, 16384, torch.bfloat16
    x, w = draw(M, K, dt, 1), draw(2 * N, K, dt, 2, 0.1)
    y, ctx = L.linear_glu_fwd(x, w, save="h")
    assert ctx.h.numel() > 1 << 31
    for lo in (0, 33000, M - 300):
        part = slice(lo, lo + 300)
        check_fwd(y[part], ctx.h[part], x[part], w, None, "silu")
    dy = torch.zeros(M, N, dtype=dt, device="cuda")
    dy[-5:] = draw(5, N, dt, 3)
    g = L.linear_glu_bwd(dy, x, w, ctx)
    check_bwd(L.LinearGluGrads(g.dx[-5:], None, None), dy[-5:], x[-5:], w, ctx.h[-5:], "silu")
    assert (g.dx[:-5] == 0).all()
    few = L.linear_glu_bwd(dy[-5:], x[-5:], w, L.LinearGluCtx(h=ctx.h[-5:]))
    assert float((few.dw.double() - g.dw.double()).norm()) <= 2 * P.half(dt) * float(g.dw.double().norm())


def test_refusals(L):
    x, w = draw(8, 64, torch.bfloat16, 1), draw(64, 64, torch.bfloat16, 2)
    with pytest.raises(ValueError, match="saved no h"):
        L.linear_glu_bwd(draw(8, 32, torch.bfloat16, 3), x, w, L.LinearGluCtx())
    with pytest.raises(TypeError, match="w is"):
        L.linear_glu_fwd(x, w.half())
    with pytest.raises(ValueError, match="bias has shape"):
        L.linear_glu_fwd(x, w, torch.zeros(32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="strides"):
        L.linear_glu_fwd(x.t().contiguous().t(), w)
    with pytest.raises(L.LnFp8Error, match="ldx"):
        L.linear_glu_fwd(draw(8, 68, torch.bfloat16, 1)[:, :64], w)
    with pytest.raises(ValueError, match="contiguous"):
        L.linear_glu_fwd(x, draw(64, 128, torch.bfloat16, 2)[:, :64])
    g = L.linear_glu_grads(8, 64, 32)
    g.workspace = g.workspace[:64]
    with pytest.raises(L.LnFp8Error, match="workspace"):
        L.linear_glu_bwd(draw(8, 32, torch.bfloat16, 3), x, w, L.LinearGluCtx(h=draw(8, 64, torch.bfloat16, 4)), grads=g)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(66, 512, 5504), (256, 2048, 5504), (333, 1024, 2736), (700, 768, 2048), (1536, 768, 1024), (1000, 1032, 2744), (300, 264, 5512)])
def test_tiles_that_are_no_power_of_two(L, M, K, N, dtype):
    """Sizes whose tiles hold 96 outputs, the last ones in part; rows behind and beside y stay as they were."""
    x, w, b = whole(M, K, dtype, 1), whole(2 * N, K, dtype, 2), whole(1, 2 * N, dtype, 3)[0]
    out = torch.full((M + 3, N + 8), 7.0, dtype=dtype, device="cuda")
    y, ctx = L.linear_glu_fwd(x, w, b, act="none", save="h", y=out[:M, :N])
    z = x.double() @ w.double().t() + b.double()
    assert torch.equal(ctx.h, z.to(dtype))
    assert torch.equal(y, (z[:, :N] * z[:, N:]).to(torch.float32).to(dtype))
    assert bool((out[M:] == 7).all()) and bool((out[:, N:] == 7).all())
    xr, wr, br = draw(M, K, dtype, 4), draw(2 * N, K, dtype, 5, 1.5 / math.sqrt(K)), draw(1, 2 * N, dtype, 6, 0.1)[0]
    for act in ACTS:
        y, ctx = L.linear_glu_fwd(xr, wr, br, act=act, save="h")
        check_fwd(y, ctx.h, xr, wr, br, act)
    L.sync_status()
