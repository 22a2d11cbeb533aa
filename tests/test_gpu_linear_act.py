"""linear_act_fwd / linear_act_bwd (GPU): products of small whole numbers bit for bit, and everything else
against the formulas in 64 bits. Products of 16-bit values are exact in fp32; an accumulation step of 16 of
them keeps at least 22 bits of the largest term, so K / 16 + 8 steps of 2^-22 of the sum of magnitudes bound a
sum over K however it is cut into pieces."""
import math

import pytest

torch = pytest.importorskip("torch")
import plain64 as P  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
# tokens, in, out: single tokens, the borders of the few-token forms, ragged and long ones
SHAPES = [(1, 64, 64), (1, 2048, 1024), (7, 72, 200), (16, 512, 136), (17, 256, 8), (33, 8, 256), (64, 640, 320), (65, 128, 128),
          (129, 200, 264), (300, 1032, 520), (513, 768, 768), (2048, 264, 1024), (700, 2048, 2056), (1500, 1800, 2056), (2600, 2568, 2560),
          (2049, 2048, 4104)]


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def draw(rows, cols, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * std + mean).to(dtype)


def whole(rows, cols, dtype, seed, most=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device="cuda").to(dtype)


def sum_error(K):
    return (K / 16 + 8) * 2.0 ** -22


def logistic_error(z, act):
    """Relative error bound of s(u): ex2.approx and rcp.approx (2 ulp each) and four roundings of u."""
    u = 1.6 * (z.abs() + 0.045 * z.abs() ** 3) if act == "gelu" else z.abs()
    return (16 + 4 * u.clamp(max=90)) * P.U


def slope_error(z, act):
    if act in ("none", "relu"):
        return torch.zeros_like(z)
    w = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3) if act == "gelu" else z
    du = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z) if act == "gelu" else torch.ones_like(z)
    s = torch.sigmoid(w)
    return 2 * logistic_error(z, act) * (s + z.abs() * s * torch.sigmoid(-w) * du) + z.abs() * du * s * P.U


def check_fwd(L, x, w, b, act, res, save):
    dt, K = x.dtype, x.shape[1]
    y, ctx = L.linear_act_fwd(x, w, b, act=act, residual=res, save=save)
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if b is not None:
        z, mag = z + b.double(), mag + b.double().abs()
    dz = sum_error(K) * mag + P.U * z.abs()
    if save == "h":
        P.assert_within(ctx.h, z, dz + P.half(dt) * (z.abs() + dz) + P.tiny(dt), "h")
    if save == "ckpt":
        nb = (z.shape[1] + 31) // 32
        top = P.blocks(z.abs() + dz).amax(2)  # the scale is of a block no larger than this
        byte = ctx.ckpt.scales[:, :nb]
        scale = torch.exp2(byte.double() - 127)
        assert (scale * P.FMAX[ctx.ckpt.dtype] >= P.blocks(z.abs() - dz).amax(2)).all()
        assert ((scale * P.FMAX[ctx.ckpt.dtype] / 2 <= top) | (byte == 0)).all()
        scale = scale.repeat_interleave(32, 1)[:, : z.shape[1]]
        tol = dz + P.HALF_CODE[ctx.ckpt.dtype] * (z.abs() + dz) + P.TINY_CODE[ctx.ckpt.dtype] * scale
        P.assert_within(P.decode(ctx.ckpt.codes, ctx.ckpt.scales, ctx.ckpt.dtype), z, tol, "checkpoint")
    want = P.act(z, act)
    tol = 1.2 * dz + logistic_error(z, act) * want.abs() + 1e-35  # no slope here passes 1.13
    if res is not None:
        want = want + res.double()
        tol = tol + P.U * want.abs()
    P.assert_within(y, want, tol + P.half(dt) * (want.abs() + tol) + P.tiny(dt), "y")
    return y, ctx


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_whole_number_products_are_exact(L, M, K, N, dtype):
    """Entries up to 3: sums stay below 2^24 and the outputs of K <= 227 columns are 16-bit exact; beyond, one rounding."""
    x, w, b, dy = whole(M, K, dtype, 1), whole(N, K, dtype, 2), whole(1, N, dtype, 3)[0], whole(M, N, dtype, 4)
    y, _ = L.linear_act_fwd(x, w, b)
    assert torch.equal(y, (x.double() @ w.double().t() + b.double()).to(dtype))
    g = L.linear_act_bwd(dy, x, w, L.LinearActCtx())
    assert torch.equal(g.dx, (dy.double() @ w.double()).to(dtype))
    assert torch.equal(g.dw, (dy.double().t() @ x.double()).to(dtype))
    assert torch.equal(g.dbias, dy.double().sum(0).float())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act,res,save", [("none", True, "none"), ("gelu", False, "ckpt"), ("gelu", True, "h"), ("relu", False, "h"),
                                          ("silu", True, "ckpt")])
def test_forward(L, M, K, N, dtype, act, res, save):
    x, w, b = draw(M, K, dtype, 1), draw(N, K, dtype, 2, 1.5 / math.sqrt(K)), draw(1, N, dtype, 3, 0.1)[0]
    check_fwd(L, x, w, b, act, draw(M, N, dtype, 4) if res else None, save)


def check_bwd(g, dy, x, dx_in, w, h, act):
    """x: the input in 64 bits, dx_in a bound of how far the kernel's 16-bit x is from it."""
    dt, (M, N), K = dy.dtype, dy.shape, w.shape[1]
    slope = P.slope(h, act) if act != "none" else torch.ones_like(dy, dtype=torch.float64)
    dz = dy.double() * slope
    e32 = dy.double().abs() * (slope_error(h, act) if act != "none" else 0) + P.U * dz.abs()
    e16 = e32 + (P.half(dt) * dz.abs() + P.tiny(dt) if act != "none" else 0)
    if g.dbias is not None:
        n = M / 600 + 8 + 8 + 608 / 8 + 8 + 40
        P.assert_within(g.dbias, dz.sum(0), n * P.U * dz.abs().sum(0) + e32.sum(0), "dbias")
    wd = w.double()
    if g.dx is not None:
        want, mag = dz @ wd, (dz.abs() + e16) @ wd.abs()
        tol = e16 @ wd.abs() + sum_error(N) * mag
        P.assert_within(g.dx, want, tol + P.half(dt) * (want.abs() + tol) + P.tiny(dt), "dx")
    if g.dw is not None:
        xa = x.abs() + dx_in
        want, mag = dz.t() @ x, (dz.abs() + e16).t() @ xa
        tol = e16.t() @ xa + dz.abs().t() @ dx_in + sum_error(M) * mag
        P.assert_within(g.dw, want, tol + P.half(dt) * (want.abs() + tol) + P.tiny(dt), "dw")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act,save,xsrc", [("none", "none", "x"), ("gelu", "ckpt", "ln"), ("silu", "h", "x"), ("relu", "ckpt", "gelu"),
                                           ("gelu", "h", "plain")])
def test_backward(L, M, K, N, dtype, act, save, xsrc):
    x, w, b = draw(M, K, dtype, 1), draw(N, K, dtype, 2, 1.5 / math.sqrt(K)), draw(1, N, dtype, 3, 0.1)[0]
    dy = draw(M, N, dtype, 5, 0.1)
    kw = {}
    if xsrc == "x":
        xin, x64, dxin = x, x.double(), torch.zeros(M, K, dtype=torch.float64, device="cuda")
    else:
        xin = L.act_ckpt_save(x)
        v = P.decode(xin.codes, xin.scales, 0)
        if xsrc == "ln":
            kw = {"x_gamma": draw(1, K, dtype, 6, 0.1, 1.0)[0], "x_beta": draw(1, K, dtype, 7, 0.1)[0]}
            x64 = v * kw["x_gamma"].double() + kw["x_beta"].double()
            dxin = (P.half(dtype) + P.U) * 1.01 * x64.abs() + P.tiny(dtype)
        else:
            kw = {"x_act": "gelu" if xsrc == "gelu" else "none"}
            x64 = P.act(v, kw["x_act"])
            dxin = (P.half(dtype) + logistic_error(v, "gelu")) * 1.01 * x64.abs() + P.tiny(dtype)
    _, ctx = L.linear_act_fwd(x, w, b, act=act, save=save)
    h = None
    if act != "none":
        h = P.decode(ctx.ckpt.codes, ctx.ckpt.scales, 0) if save == "ckpt" else ctx.h.double()
    g = L.linear_act_bwd(dy, xin, w, ctx, **kw)
    check_bwd(g, dy, x64, dxin, w, h, act)
    again = L.linear_act_bwd(dy, xin, w, ctx, **kw)
    assert torch.equal(g.dx, again.dx) and torch.equal(g.dw, again.dw) and torch.equal(g.dbias, again.dbias)


def test_checkpoint_formats(L):
    x, w, dy = draw(40, 128, torch.bfloat16, 1), draw(96, 128, torch.bfloat16, 2, 0.1), draw(40, 96, torch.bfloat16, 3)
    y, ctx = L.linear_act_fwd(x, w, act="gelu", save="ckpt", ctx=L.LinearActCtx(ckpt=L.act_ckpt(40, 96, dtype=L.E5M2)))
    z = x.double() @ w.double().t()
    scale = torch.exp2(ctx.ckpt.scales[:, :3].double() - 127).repeat_interleave(32, 1)
    P.assert_within(P.decode(ctx.ckpt.codes, ctx.ckpt.scales, 1), z, P.HALF_CODE[1] * 1.001 * z.abs() + P.TINY_CODE[1] * scale
                    + sum_error(128) * (x.double().abs() @ w.double().abs().t()), "E5M2 checkpoint")
    xck = L.act_ckpt_save(x, dtype=L.E5M2)
    g = L.linear_act_bwd(dy, xck, w, ctx)
    v = P.decode(xck.codes, xck.scales, 1)
    check_bwd(g, dy, v, P.half(torch.bfloat16) * v.abs(), w, P.decode(ctx.ckpt.codes, ctx.ckpt.scales, 1), "gelu")


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_backward_against_differences(L, act):
    """The 64-bit loss sum(dy y) along random directions: central differences against the kernels' gradients, which
    are 16-bit: half a step of each gradient (and of dz inside it) times the direction bounds the difference."""
    M, K, N, dt = 24, 64, 40, torch.float16
    x, w, b, dy = draw(M, K, dt, 1), draw(N, K, dt, 2, 0.1), draw(1, N, dt, 3)[0], draw(M, N, dt, 4)
    ctx = L.LinearActCtx(act=act)
    if act != "none":
        ctx.h = (x.double() @ w.double().t() + b.double()).to(dt)
    g = L.linear_act_bwd(dy, x, w, ctx)

    def loss(X, W, B):
        return float((P.act(X @ W.t() + B, act) * dy.double()).sum())

    h64 = x.double() @ w.double().t() + b.double()
    dz = dy.double() * P.slope(h64, act)
    # dz carries h's rounding (no second derivative here passes 1.3) and its own
    edz = dy.double().abs() * 1.3 * P.half(dt) * h64.abs() * (act != "none") + 2 * P.half(dt) * dz.abs() + P.tiny(dt)
    for seed in range(3):
        vx, vw, vb = draw(M, K, dt, 30 + seed).double(), draw(N, K, dt, 40 + seed).double(), draw(1, N, dt, 50 + seed).double()
        e = 1e-5
        num = (loss(x.double() + e * vx, w.double() + e * vw, b.double() + e * vb)
               - loss(x.double() - e * vx, w.double() - e * vw, b.double() - e * vb)) / (2 * e)
        ana = float((g.dx.double() * vx).sum() + (g.dw.double() * vw).sum() + (g.dbias.double() * vb[0]).sum())
        tol = ((edz @ w.double().abs() + P.half(dt) * g.dx.double().abs()) * vx.abs()).sum() \
            + ((edz.t() @ x.double().abs() + P.half(dt) * g.dw.double().abs()) * vw.abs()).sum() + (edz.sum(0) * vb[0].abs()).sum()
        assert abs(num - ana) <= float(tol) * 1.01 + 1e-6 * abs(num)


@pytest.mark.parametrize("M,K,N", [(5, 128, 64), (300, 192, 264), (600, 512, 520)])
def test_strides_and_neighbours(L, M, K, N):
    """Rows inside wider tensors (a slice of a fused QKV output, say); what lies around the outputs stays."""
    dt = torch.bfloat16
    x, r, dy = (draw(M, c + 40, dt, s)[:, 16 : 16 + c] for c, s in ((K, 1), (N, 2), (N, 3)))
    w, b = draw(N, K, dt, 4, 0.1), draw(1, N, dt, 5)[0]
    buf = torch.full((M + 2, N + 40), 7.0, dtype=dt, device="cuda")
    y = buf[1 : M + 1, 24 : 24 + N]
    _, ctx = L.linear_act_fwd(x, w, b, act="gelu", residual=r, save="ckpt", y=y)
    want, wctx = L.linear_act_fwd(x.contiguous(), w, b, act="gelu", residual=r.contiguous(), save="ckpt")
    assert torch.equal(y, want) and torch.equal(ctx.ckpt.codes, wctx.ckpt.codes)
    y.fill_(7.0)
    assert (buf == 7.0).all()
    g = L.linear_act_grads(M, K, N, act="gelu")
    wide = torch.full((M + 2, K + 40), 7.0, dtype=dt, device="cuda")
    g.dx = wide[1 : M + 1, 8 : 8 + K]
    L.linear_act_bwd(dy, x, w, ctx, grads=g)
    want = L.linear_act_bwd(dy.contiguous(), x.contiguous(), w, ctx)
    assert torch.equal(g.dx, want.dx) and torch.equal(g.dw, want.dw) and torch.equal(g.dbias, want.dbias)
    g.dx.fill_(7.0)
    assert (wide == 7.0).all()
    g = L.linear_act_bwd(dy, x, w, L.LinearActCtx())
    want = L.linear_act_bwd(dy.contiguous(), x.contiguous(), w, L.LinearActCtx())
    assert torch.equal(g.dx, want.dx) and torch.equal(g.dw, want.dw) and torch.equal(g.dbias, want.dbias)


def test_offsets_past_32_bits(L):
    """2.2e9 elements of y, h and dz: the last rows as those of a call of their own (whole numbers: no order matters)."""
    M, K, N, tail = 270001, 64, 8192, 300
    x, w = whole(M, K, torch.bfloat16, 1), whole(N, K, torch.bfloat16, 2)
    y, ctx = L.linear_act_fwd(x, w, act="relu", save="ckpt")
    y2, ctx2 = L.linear_act_fwd(x[-tail:], w, act="relu", save="ckpt")
    assert torch.equal(y[-tail:], y2) and torch.equal(ctx.ckpt.codes[-tail:], ctx2.ckpt.codes)
    assert torch.equal(ctx.ckpt.scales[-tail:], ctx2.ckpt.scales)
    del y, y2
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dy[-tail:] = whole(tail, N, torch.bfloat16, 3)
    g = L.linear_act_bwd(dy, x, w, ctx)
    g2 = L.linear_act_bwd(dy[-tail:], x[-tail:], w, ctx2)
    assert torch.equal(g.dx[-tail:], g2.dx) and not g.dx[:-tail].any()
    assert torch.equal(g.dw, g2.dw) and torch.equal(g.dbias, g2.dbias)
    L.sync_status()


def test_some_gradients_only(L):
    """What is not asked for is left out. How many pieces K is cut into depends on which products a launch holds, so
    a gradient asked for alone is another sum of the same terms: each is within sum_error of the exact one and half
    a step of the type from that, and the two within twice that of one another. dbias is the same sum."""
    M, K, N = 200, 128, 192
    x, w, dy = draw(M, K, torch.bfloat16, 1), draw(N, K, torch.bfloat16, 2, 0.1), draw(M, N, torch.bfloat16, 3)
    full = L.linear_act_bwd(dy, x, w, L.LinearActCtx())
    d = dy.double()
    bound = {"dx": sum_error(N) * (d.abs() @ w.double().abs()), "dw": sum_error(M) * (d.abs().t() @ x.double().abs()), "dbias": 0}
    for keep in ("dx", "dw", "bias"):
        g = L.linear_act_grads(M, K, N, **{k: k == keep for k in ("dx", "dw", "bias")})
        L.linear_act_bwd(dy, x if keep == "dw" else None, w, L.LinearActCtx(), grads=g)
        name = "dbias" if keep == "bias" else keep
        want = getattr(full, name).double()
        P.assert_within(getattr(g, name), want, 2 * (bound[name] + P.half(torch.bfloat16) * (want.abs() + bound[name])) * (name != "dbias"), name)
        assert sum(v is not None for v in (g.dx, g.dw, g.dbias)) == 1
    assert L.linear_act_bwd(dy, None, w, L.LinearActCtx()).dw is None


def test_no_tokens(L):
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), draw(32, 64, torch.bfloat16, 1)
    y, ctx = L.linear_act_fwd(x, w, act="gelu", save="ckpt")
    g = L.linear_act_bwd(y, x, w, ctx)
    assert y.shape == (0, 32) and g.dx.shape == (0, 64) and not g.dw.any() and not g.dbias.any()


def test_nan_and_inf_stay_in_their_rows(L):
    for M in (4, 200):
        x, w = draw(M, 128, torch.bfloat16, 1), draw(64, 128, torch.bfloat16, 2)
        x[1, 3], x[2, 5] = float("nan"), float("inf")
        y, ctx = L.linear_act_fwd(x, w, act="silu", save="ckpt")
        keep = [i for i in range(M) if i not in (1, 2)]
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any() and torch.isfinite(y[keep]).all()
        back = L.act_ckpt_restore(ctx.ckpt)
        assert torch.isnan(back[1:3]).all() and torch.isfinite(back[keep]).all()


# few tiles over a long K forward; few tiles of a weight gradient over many tokens, ragged
LONG = [(200, 4096, 1000), (300, 4104, 520), (9001, 520, 264), (5000, 776, 520)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", LONG)
def test_products_cut_along_their_sums(L, M, K, N, dtype):
    test_whole_number_products_are_exact(L, M, K, N, dtype)
    test_forward(L, M, K, N, dtype, "gelu", True, "ckpt")
    test_forward(L, M, K, N, dtype, "none", False, "none")
    for xsrc in ("x", "ln"):
        test_backward(L, M, K, N, dtype, "gelu", "ckpt", xsrc)


@pytest.mark.parametrize("act", ["gelu", "relu", "silu"])
def test_nan_pre_activations_reach_the_gradients(L, act):
    """A pre-activation that was NaN, or whose checkpoint block holds an Inf, must not pass for a zero slope."""
    for M in (8, 300):
        h = draw(M, 64, torch.bfloat16, 1)
        h[1, 3], h[2, 40] = float("nan"), float("inf")
        ck = L.act_ckpt_save(h)
        dy, w = torch.ones_like(h), torch.eye(64, dtype=torch.bfloat16, device="cuda")
        g = L.linear_act_bwd(dy, h, w, L.LinearActCtx(act=act, h=h))
        assert torch.isnan(g.dbias[3]) and torch.isnan(g.dx[1]).all() and torch.isfinite(g.dx[3:]).all()
        g = L.linear_act_bwd(dy, h, w, L.LinearActCtx(act=act, ckpt=ck))
        assert torch.isnan(g.dbias).all() and torch.isnan(g.dx[1:3]).all() and torch.isfinite(g.dx[3:]).all()


def test_far_out_pre_activations(L):
    """Slopes and values where e^-u and z^2 leave fp32."""
    h = torch.tensor([[0.0, -0.0, 20.0, -20.0, 1e4, -1e4, 1e20, -1e20] * 2], dtype=torch.bfloat16, device="cuda")
    dy, w = torch.ones_like(h), torch.eye(16, dtype=torch.bfloat16, device="cuda")
    for act in ("gelu", "silu", "relu"):
        y, _ = L.linear_act_fwd(h, w, act=act)
        want = P.act(h.double(), act)
        P.assert_within(y, want, P.half(torch.bfloat16) * 1.01 * want.abs() + 1e-30, act)
        g = L.linear_act_bwd(dy, h, w, L.LinearActCtx(act=act, h=h))
        want = P.slope(h.double().clamp(-1e5, 1e5), act)
        # at -20, silu' = s (1 - 19): s is (16 + 4 * 20) U off, 21 / 19 of it and as much again in 1 - s
        P.assert_within(g.dbias[None], want, 2e-5 * want.abs() + 1e-30, act)


def test_stream_and_graph(L):
    x, w, dy = draw(300, 256, torch.bfloat16, 1), draw(512, 256, torch.bfloat16, 2, 0.1), draw(300, 512, torch.bfloat16, 3)

    def step(stream=None):
        y, ctx = L.linear_act_fwd(x, w, act="gelu", save="ckpt", stream=stream)
        g = L.linear_act_bwd(dy, x, w, ctx, stream=stream)
        return y, g.dx, g.dw, g.dbias

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    x.copy_(draw(300, 256, torch.bfloat16, 9))
    gr.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    L.sync_status()


def test_binding_refuses_workspaces_it_cannot_use(L):
    x, w = draw(8, 64, torch.bfloat16, 1), draw(32, 64, torch.bfloat16, 2)
    dy = draw(8, 32, torch.bfloat16, 3)
    for ws, err in ((torch.empty(1 << 20, dtype=torch.uint8), TypeError),
                    (torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20), ValueError)):
        g = L.linear_act_grads(8, 64, 32)
        g.workspace = ws
        with pytest.raises(err, match="workspace"):
            L.linear_act_bwd(dy, x, w, L.LinearActCtx(), grads=g)


def test_binding_refuses(L):
    x, w = draw(8, 64, torch.bfloat16, 1), draw(32, 64, torch.bfloat16, 2)
    for call in (lambda: L.linear_act_fwd(x.float(), w.float()), lambda: L.linear_act_fwd(x, w.half()), lambda: L.linear_act_fwd(x.cpu(), w)):
        with pytest.raises(TypeError):
            call()
    y, ctx = L.linear_act_fwd(x, w, act="gelu")
    for call in (lambda: L.linear_act_fwd(x, w, act="tanh"), lambda: L.linear_act_fwd(x, w, save="all"), lambda: L.linear_act_fwd(x, w[:, :32]),
                 lambda: L.linear_act_fwd(x, w, residual=x), lambda: L.linear_act_bwd(y, x, w, ctx), lambda: L.linear_act_bwd(y, x[:4], w, L.LinearActCtx()),
                 lambda: L.linear_act_fwd(x[:1].expand(8, 64), w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: L.linear_act_fwd(x[:, 4:60].contiguous()[:, :52], w[:, :52].contiguous()),
                 lambda: L.linear_act_bwd(y, x, w, L.LinearActCtx(), x_act="gelu")):
        with pytest.raises(L.LnFp8Error):
            call()


NAN_ROWS = [8, 64, 300, 2048]  # few tokens, tokens on the columns, tiles of one and of several rounds


def near_eight(N, cols):
    """The other columns of the groups of eight that hold `cols`, and all columns outside those groups."""
    eight = sorted({8 * (c // 8) + i for c in cols for i in range(8)} - set(cols))
    return eight, [i for i in range(N) if i not in eight and i not in cols]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
@pytest.mark.parametrize("where", ["w", "bias", "bias beside a far one"])
@pytest.mark.parametrize("M", NAN_ROWS)
def test_a_nan_feature_stays_in_its_column(L, M, where, act, dtype):
    """A NaN in one row of w, or in one entry of the bias, makes that column NaN and no other. The activation of the other
    columns of its group of eight may be computed in another way: both are within logistic_error of the exact value, and
    half a step of the type. All other columns are the same bits."""
    K, N, bad = 256, 776, [37, 100, 775]
    x, w, b = draw(M, K, dtype, 1), draw(N, K, dtype, 2, 1.5 / math.sqrt(K)), draw(1, N, dtype, 3, 0.1)[0]
    if where == "bias beside a far one":
        b[[c ^ 1 for c in bad]] = -1000.0
    y0, ctx0 = L.linear_act_fwd(x, w, b, act=act, save="h")
    if where == "w":
        w[bad, 5] = math.nan
    else:
        b[bad] = math.nan
    y, ctx = L.linear_act_fwd(x, w, b, act=act, save="h")
    near, rest = near_eight(N, bad)
    assert torch.isnan(y[:, bad]).all() and torch.isnan(ctx.h[:, bad]).all()
    assert torch.equal(ctx.h[:, near + rest], ctx0.h[:, near + rest]) and torch.equal(y[:, rest], y0[:, rest])
    v = y0[:, near].double()
    err = logistic_error(ctx0.h[:, near].double() * (1 + P.half(dtype)), act) if act != "relu" else 0
    P.assert_within(y[:, near], v, (2 * err + 2 * P.half(dtype)) * 1.01 * v.abs() + 2 * P.tiny(dtype), "columns beside the NaN")
    L.sync_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("M", NAN_ROWS)
def test_a_nan_pre_activation_stays_in_its_column(L, M, far, act, dtype):
    """One NaN of h makes its column's dbias and dw NaN, its row's dx, and nothing else. The slopes of its group of eight
    may be computed in another way, each within slope_error; beside it a value whose e^-u leaves fp32."""
    K, N, r, c = 136, 264, M - 2, 101
    x, w, h, dy = draw(M, K, dtype, 1), draw(N, K, dtype, 2, 0.1), draw(M, N, dtype, 3), draw(M, N, dtype, 4, 0.1)
    if far:
        h[r, c ^ 1] = -100.0
    g0 = L.linear_act_bwd(dy, x, w, L.LinearActCtx(act=act, h=h))
    clean = h.double()
    h = h.clone()
    h[r, c] = math.nan
    g = L.linear_act_bwd(dy, x, w, L.LinearActCtx(act=act, h=h))
    near, rest = near_eight(N, [c])
    assert torch.isnan(g.dbias[c]) and torch.isnan(g.dw[c]).all() and torch.isnan(g.dx[r]).all()
    rows = [i for i in range(M) if i != r]
    assert torch.equal(g.dx[rows], g0.dx[rows]) and torch.equal(g.dbias[rest], g0.dbias[rest]) and torch.equal(g.dw[rest], g0.dw[rest])
    # the row's terms of these columns move by twice the slope's error, and as operands by a step of the type more
    dz = dy.double().abs() * P.slope(clean, act).abs()
    e = 2 * dy[r, near].double().abs() * (slope_error(clean[r, near], act) + P.U)
    n = M / 600 + 8 + 8 + 608 / 8 + 8 + 40
    P.assert_within(g.dbias[near], g0.dbias[near].double(), e + 2 * n * P.U * dz[:, near].sum(0), "dbias")
    e16 = e + 2 * P.half(dtype) * dz[r, near] + 2 * P.tiny(dtype)
    v = g0.dw[near].double()
    tol = e16[:, None] * x[r].double().abs() + 2 * sum_error(M) * (dz[:, near].t() @ x.double().abs())
    P.assert_within(g.dw[near], v, 1.01 * tol + 2 * P.half(dtype) * (v.abs() + 1.01 * tol) + 2 * P.tiny(dtype), "dw")
    L.sync_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("std", [1.0, 1e-3])
@pytest.mark.parametrize("M,K,N", [(64, 72, 200), (300, 264, 136), (2049, 520, 264), (9001, 520, 264)])
def test_weight_gradient_of_normalised_rows_does_not_round_x(L, M, K, N, std, dtype):
    """dw of x = v gamma + beta: the product reads v, exactly in bf16 and within half a step of fp16's subnormals, and x is
    never formed. Left are the products' and the column sums' fp32 roundings, of v gamma and beta apart, and dw's own."""
    xck = L.act_ckpt_save(draw(M, K, dtype, 1, std))
    w, dy = draw(N, K, dtype, 2, 0.1), draw(M, N, dtype, 3, 0.1)
    gamma, beta = draw(1, K, dtype, 4, 0.1, 1.0)[0], draw(1, K, dtype, 5, 0.1 * std)[0]
    g = L.linear_act_bwd(dy, xck, w, L.LinearActCtx(), x_gamma=gamma, x_beta=beta)
    v, d, ga, be = P.decode(xck.codes, xck.scales, 0), dy.double(), gamma.double(), beta.double()
    want = d.t() @ (v * ga + be)
    tol = (sum_error(M) + 4 * P.U) * (d.abs().t() @ (v.abs() * ga.abs() + be.abs()))
    if dtype == torch.float16:
        tol = tol + d.abs().sum(0)[:, None] * ga.abs() * P.tiny(dtype)
    tol = 1.01 * tol
    P.assert_within(g.dw, want, tol + P.half(dtype) * (want.abs() + tol) + P.tiny(dtype), "dw")


def test_restored_inputs_saturate_at_the_types_largest_value(L):
    """A checkpoint's values enter the products in the products' type: beyond 65504 fp16 holds 65504, gamma or not."""
    x = torch.full((40, 32), 1e6, device="cuda")
    x[:, :16] = -1e6
    xck, w = L.act_ckpt_save(x), torch.zeros(8, 32, dtype=torch.float16, device="cuda")
    dy = torch.full((40, 8), 2.0 ** -10, dtype=torch.float16, device="cuda")
    sign = x[0].sign()
    one, zero = torch.full_like(w[0], 0.125), torch.zeros_like(w[0])
    assert torch.equal(L.linear_act_bwd(dy, xck, w, L.LinearActCtx()).dw[3], (40 * 2.0 ** -10 * 65504 * sign).half())
    g = L.linear_act_bwd(dy, xck, w, L.LinearActCtx(), x_gamma=one, x_beta=zero)
    assert torch.equal(g.dw[3], (40 * 2.0 ** -13 * 65504 * sign).half())


# a few tokens: K long enough for one, two, four and eight warps to a row, whole and ragged pieces; and outputs that are
# too many for that form
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(1, 1000, 5000), (3, 2056, 2000), (2, 4104, 1032), (4, 8192, 264), (1, 16392, 136), (3, 12280, 16),
                                   (2, 264, 8200), (4, 1032, 2568), (3, 4104, 4104)])
def test_a_few_tokens_over_long_rows(L, M, K, N, dtype):
    x, w, b = whole(M, K, dtype, 1), whole(N, K, dtype, 2), whole(1, N, dtype, 3)[0]
    assert torch.equal(L.linear_act_fwd(x, w, b)[0], (x.double() @ w.double().t() + b.double()).to(dtype))
    x, w, b = draw(M, K, dtype, 1), draw(N, K, dtype, 2, 1.5 / math.sqrt(K)), draw(1, N, dtype, 3, 0.1)[0]
    check_fwd(L, x, w, b, "gelu", draw(M, N, dtype, 4), "h")


# the last number of tokens whose bias sums come from one launch, and the next: without an activation small and large
# weights, with one
@pytest.mark.parametrize("M,K,N,act,save,xsrc", [(m, K, N, act, save, xsrc) for lo, K, N, act, save, xsrc in
                                                 [(1024, 768, 776, "none", "none", "x"), (512, 1544, 1032, "none", "none", "ln"),
                                                  (320, 264, 520, "gelu", "ckpt", "ln"), (320, 136, 264, "silu", "h", "x")] for m in (lo, lo + 1)])
def test_backward_on_both_sides_of_the_one_launch_sums(L, M, K, N, act, save, xsrc):
    test_backward(L, M, K, N, torch.bfloat16, act, save, xsrc)
    if act == "none":
        test_whole_number_products_are_exact(L, M, K, N, torch.bfloat16)
