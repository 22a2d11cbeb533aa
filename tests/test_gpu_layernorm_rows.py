"""layernorm_fwd / layernorm_bwd (GPU) against the formulas in 64 bits. Tolerances count roundings: half a
step of the output type, and U = 2^-24 per fp32 step. A row sum in fp32 goes through at most 16 terms
in a thread, 5 shuffles and 32 warps' partials: 30 U of the sum of magnitudes bounds it."""
import pytest

torch = pytest.importorskip("torch")
import plain64 as P  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 2048), (1, 1), (3, 7), (257, 768), (40, 1000), (33, 1001), (5, 2050), (19, 4096), (7, 8192), (3, 16384),
          (2, 16381), (1000, 64), (700, 520)]


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def draw(rows, cols, dtype, seed, std=1.0, mean=0.0, outliers=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(rows, cols, generator=g, device="cuda") * std + mean
    if outliers:
        v = torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 1e-3, v * 50, v)
    return v.to(dtype)


def params(cols, dtype):
    return draw(1, cols, dtype, 91, 0.1, 1.0)[0], draw(1, cols, dtype, 92, 0.1)[0]


def stats(h, eps=1e-5):
    v = h.double()
    mu = v.mean(1)
    rs = ((v - mu[:, None]).square().mean(1) + eps) ** -0.5
    return mu, rs, (v - mu[:, None]) * rs[:, None]


def xhat_error(h, rs, xh):
    """|error| of the fp32 normalised rows: the mean's (30 U of the mean magnitude), the subtraction's and rs's.
    The centred squares' sum (30 U), / D, + eps, sqrt and 1/x are 34 U on the square, 17 on rs, and the mean's own
    error enters the squares only in second order; the subtraction and the product are 2 more, 20 in all."""
    return 30 * P.U * h.double().abs().mean(1, keepdim=True) * rs[:, None] + 20 * P.U * xh.abs()


def check_fwd(y, ctx, h, gamma, beta):
    mu, rs, xh = stats(h)
    dxh = xhat_error(h, rs, xh)
    g, b = gamma.double(), beta.double()
    want = xh * g + b
    P.assert_within(ctx.mu, mu, 31 * P.U * h.double().abs().mean(1), "mu")
    # a constant row: the squares are those of the mean's own error
    slack = (30 * P.U * h.double().abs().mean(1)) ** 2 * rs ** 3
    P.assert_within(ctx.rsigma, rs, 20 * P.U * rs + slack, "rsigma")
    tol = g.abs() * (dxh + slack[:, None] * (h.double() - mu[:, None]).abs()) + 2 * P.U * want.abs()
    P.assert_within(y, want, tol * 1.01 + P.half(y.dtype) * want.abs() + P.tiny(y.dtype), "y")
    if ctx.ckpt is not None:
        fmt = ctx.ckpt.dtype
        lo, hi = P.scale_bytes(xh * (1 - 1e-5), fmt), P.scale_bytes(xh * (1 + 1e-5), fmt)
        byte = ctx.ckpt.scales[:, : lo.shape[1]]
        assert ((byte == lo) | (byte == hi)).all()
        scale = torch.exp2(byte.double() - 127).repeat_interleave(32, 1)[:, : h.shape[1]]
        tol = dxh * 1.1 + P.HALF_CODE[fmt] * xh.abs() + P.TINY_CODE[fmt] * scale
        P.assert_within(P.decode(ctx.ckpt.codes, ctx.ckpt.scales, fmt), xh, tol, "checkpoint")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("res,ckpt", [(False, False), (True, True), (False, True)])
def test_forward(L, rows, cols, dtype, res, ckpt):
    x = draw(rows, cols, dtype, 1, outliers=True)
    r = draw(rows, cols, dtype, 2) if res else None
    gamma, beta = params(cols, dtype)
    y, ctx = L.layernorm_fwd(x, gamma, beta, residual=r, ckpt=ckpt)
    if res:
        h = (x.float() + r.float()).to(dtype)  # the fp32 sum of two 16-bit values rounds the same way once more
        assert torch.equal(ctx.x, h)
    check_fwd(y, ctx, ctx.x, gamma, beta)


@pytest.mark.parametrize("dtype", DTYPES)
def test_forward_large_mean_constant_rows_and_eps(L, dtype):
    gamma, beta = params(768, dtype)
    x = draw(64, 768, dtype, 3, std=0.5, mean=100.0)
    x[7] = 100.0
    x[8] = 0.0
    y, ctx = L.layernorm_fwd(x, gamma, beta, ckpt=True)
    check_fwd(y, ctx, x, gamma, beta)
    y, ctx = L.layernorm_fwd(x[:5], gamma, beta, eps=0.5)
    _, rs, _ = stats(x[:5], 0.5)
    P.assert_within(ctx.rsigma, rs, 21 * P.U * rs, "rsigma")


@pytest.mark.parametrize("fmt", [0, 1])
def test_forward_checkpoint_formats_and_param_types(L, fmt):
    for pd in DTYPES:
        gamma, beta = params(520, pd)
        x = draw(33, 520, torch.bfloat16, 4)
        y, ctx = L.layernorm_fwd(x, gamma, beta, ckpt=L.act_ckpt(33, 520, dtype=fmt))
        check_fwd(y, ctx, x, gamma, beta)


def check_bwd(g, dy, xh, dxh, rs, gamma, dres):
    """xh: the normalised rows the backward used (64 bits), dxh the bound of their fp32 error."""
    d, rows = dy.double(), dy.shape[0]
    gg = d * gamma.double()
    mg, mx = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    want = rs[:, None] * (gg - mg - xh * mx)
    tol = rs[:, None] * (34 * P.U * gg.abs().mean(1, keepdim=True) + 6 * P.U * gg.abs() + dxh * mx.abs() +
                         xh.abs() * (36 * P.U * (gg * xh).abs().mean(1, keepdim=True) + (gg.abs() * dxh).mean(1, keepdim=True)))
    tol = tol * 1.01 + 3 * P.U * want.abs()
    if dres is not None:
        want = want + dres.double()
        tol = tol + P.U * want.abs()
    P.assert_within(g.dx, want, tol + P.half(g.dx.dtype) * want.abs() + P.tiny(g.dx.dtype), "dx")
    # column sums: at most rows / 256 + 8 rows in a thread, then 16 groups and 64 partial rows a warp, 8 warps
    n = (rows // 256 + 8) + 90
    P.assert_within(g.dgamma, (d * xh).sum(0), n * P.U * (d * xh).abs().sum(0) + (d.abs() * dxh).sum(0), "dgamma")
    P.assert_within(g.dbeta, d.sum(0), n * P.U * d.abs().sum(0), "dbeta")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("ckpt,res", [(False, False), (True, True), (False, True)])
def test_backward(L, rows, cols, dtype, ckpt, res):
    x = draw(rows, cols, dtype, 1, outliers=True)
    gamma, beta = params(cols, dtype)
    dy = draw(rows, cols, dtype, 5, 0.1)
    dres = draw(rows, cols, dtype, 6, 0.1) if res else None
    _, ctx = L.layernorm_fwd(x, gamma, beta, ckpt=ckpt)
    g = L.layernorm_bwd(dy, ctx, gamma, dresidual=dres)
    rs = ctx.rsigma.double()
    if ckpt:
        xh = P.decode(ctx.ckpt.codes, ctx.ckpt.scales, 0)
        dxh = torch.zeros_like(xh)
    else:
        xh = (x.double() - ctx.mu.double()[:, None]) * rs[:, None]
        dxh = 2.01 * P.U * xh.abs()
    check_bwd(g, dy, xh, dxh, rs, gamma, dres)
    again = L.layernorm_bwd(dy, ctx, gamma, dresidual=dres)
    for a, b in ((g.dx, again.dx), (g.dgamma, again.dgamma), (g.dbeta, again.dbeta)):
        assert torch.equal(a, b)


# rows of a few lanes (a head's columns), the last of a block's row groups without one, rings that turn more than once;
# and rows wide enough to keep their column sums elsewhere, several to a block
MORE = [(1, 8), (33, 16), (70, 24), (100, 64), (259, 72), (131, 128), (70, 136), (133, 200), (1000, 256), (40000, 64), (12001, 128),
        (700, 9001), (640, 16384)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", MORE)
@pytest.mark.parametrize("res,ckpt", [(False, False), (True, True), (False, True)])
def test_narrow_and_wide_rows(L, rows, cols, dtype, res, ckpt):
    test_forward(L, rows, cols, dtype, res, ckpt)
    test_backward(L, rows, cols, dtype, ckpt, res)


@pytest.mark.parametrize("rows,cols", [(9, 64), (6, 77)])
def test_backward_against_differences(L, rows, cols):
    """fp32 gradients against central differences of the 64-bit forward: step 1e-5 leaves 1e-9 of truncation,
    the fp32 gradients 64 U of the magnitudes summed."""
    x, dy = draw(rows, cols, torch.float32, 7), draw(rows, cols, torch.float32, 8)
    gamma, beta = params(cols, torch.float32)
    _, ctx = L.layernorm_fwd(x, gamma, beta)
    g = L.layernorm_bwd(dy, ctx, gamma)

    def loss(v, ga, be):
        return float(((stats(v)[2] * ga + be) * dy.double()).sum())

    for seed in range(3):
        vx, vg, vb = (draw(*s, torch.float32, 20 + seed).double() for s in ((rows, cols), (1, cols), (1, cols)))
        e = 1e-5
        num = (loss(x.double() + e * vx, gamma.double() + e * vg[0], beta.double() + e * vb[0])
               - loss(x.double() - e * vx, gamma.double() - e * vg[0], beta.double() - e * vb[0])) / (2 * e)
        parts = [(g.dx.double() * vx), (g.dgamma.double() * vg[0]), (g.dbeta.double() * vb[0])]
        ana = float(sum(p.sum() for p in parts))
        assert abs(num - ana) <= 1e-6 * float(sum(p.abs().sum() for p in parts))


def test_no_rows_and_one_column(L):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gamma, beta = params(64, torch.bfloat16)
    y, ctx = L.layernorm_fwd(x, gamma, beta, ckpt=True)
    g = L.layernorm_bwd(x, ctx, gamma)
    assert y.shape == (0, 64) and not g.dgamma.any() and not g.dbeta.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lo,cols", [(0, 136), (8, 128), (1, 130), (3, 64)])
def test_strides_alignment_and_neighbours(L, dtype, lo, cols):
    """Rows inside wider tensors, from an odd column on, give what contiguous copies give; the rest stays."""
    a, b, c = (draw(40, 200, dtype, s)[:, lo : lo + cols] for s in (1, 2, 3))
    gamma, beta = params(cols, dtype)
    buf = torch.full((42, 200), 7.0, dtype=dtype, device="cuda")
    y = buf[1:41, lo : lo + cols]
    _, ctx = L.layernorm_fwd(a, gamma, beta, residual=b, ckpt=True, y=y)
    check_fwd(y, ctx, (a.float() + b.float()).to(dtype), gamma, beta)
    g = L.layernorm_grads(40, cols, dtype=dtype)
    g.dx = y
    L.layernorm_bwd(c, L.LayerNormCtx(a, ctx.mu, ctx.rsigma), gamma, dresidual=b, grads=g)
    want = L.layernorm_bwd(c.contiguous(), L.LayerNormCtx(a.contiguous(), ctx.mu, ctx.rsigma), gamma, dresidual=b.contiguous())
    xh = (a.double() - ctx.mu.double()[:, None]) * ctx.rsigma.double()[:, None]
    check_bwd(g, c, xh, 2.01 * P.U * xh.abs(), ctx.rsigma.double(), gamma, b)
    check_bwd(want, c, xh, 2.01 * P.U * xh.abs(), ctx.rsigma.double(), gamma, b)
    y.fill_(7.0)
    assert (buf == 7.0).all()


def test_offsets_past_32_bits(L):
    rows, cols = 132000, 16384
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = draw(2, cols, torch.bfloat16, 3)
    x[-2:] = tail
    gamma, beta = params(cols, torch.bfloat16)
    y, ctx = L.layernorm_fwd(x, gamma, beta, ckpt=True)
    y2, ctx2 = L.layernorm_fwd(tail, gamma, beta, ckpt=True)
    assert torch.equal(y[-2:], y2) and torch.equal(ctx.ckpt.codes[-2:], ctx2.ckpt.codes)
    g = L.layernorm_bwd(x, ctx, gamma)
    g2 = L.layernorm_bwd(tail, ctx2, gamma)
    assert torch.equal(g.dx[-2:], g2.dx) and not g.dx[:-2].any()


def test_nan_and_inf_stay_in_their_rows(L):
    x = draw(16, 768, torch.bfloat16, 2)
    x[3, 5], x[7, 1] = float("nan"), float("inf")
    gamma, beta = params(768, torch.bfloat16)
    y, ctx = L.layernorm_fwd(x, gamma, beta, ckpt=True)
    keep = [i for i in range(16) if i not in (3, 7)]
    assert torch.isnan(y[3]).all() and torch.isnan(y[7]).all() and torch.isfinite(y[keep]).all()
    back = L.act_ckpt_restore(ctx.ckpt)
    assert torch.isnan(back[3]).all() and torch.isnan(back[7]).all() and torch.isfinite(back[keep]).all()


def test_stream_and_graph(L):
    x, dy = draw(300, 768, torch.bfloat16, 4), draw(300, 768, torch.bfloat16, 5)
    gamma, beta = params(768, torch.bfloat16)

    def step(stream=None):
        y, ctx = L.layernorm_fwd(x, gamma, beta, residual=dy, ckpt=True, stream=stream)
        g = L.layernorm_bwd(y, ctx, gamma, dresidual=dy, stream=stream)
        return g.dx, g.dgamma, g.dbeta

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    x.copy_(draw(300, 768, torch.bfloat16, 9))
    gr.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_binding_refuses_workspaces_it_cannot_use(L):
    x = draw(4, 64, torch.bfloat16, 1)
    gamma, beta = params(64, torch.bfloat16)
    _, ctx = L.layernorm_fwd(x, gamma, beta)
    for ws, err in ((torch.empty(1 << 20, dtype=torch.uint8), TypeError),
                    (torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20), ValueError)):
        g = L.layernorm_grads(4, 64)
        g.workspace = ws
        with pytest.raises(err, match="workspace"):
            L.layernorm_bwd(x, ctx, gamma, grads=g)


def test_binding_refuses(L):
    x = draw(4, 64, torch.bfloat16, 1)
    gamma, beta = params(64, torch.bfloat16)
    _, ctx = L.layernorm_fwd(x, gamma, beta)
    for bad in (dict(x=x.cpu()), dict(x=x.double())):
        with pytest.raises(TypeError):
            L.layernorm_fwd(bad["x"], gamma, beta)
    for kw in (dict(residual=x.float()), dict(beta=beta.float())):
        with pytest.raises(TypeError):
            L.layernorm_fwd(x, gamma, kw.get("beta", beta), residual=kw.get("residual"))
    for call in (lambda: L.layernorm_fwd(x[0], gamma, beta), lambda: L.layernorm_fwd(x, gamma[:5], beta[:5]),
                 lambda: L.layernorm_fwd(x[:, ::2], gamma[::2].contiguous(), beta[::2].contiguous()),
                 lambda: L.layernorm_bwd(x[:1].expand(4, 64), ctx, gamma), lambda: L.layernorm_bwd(x[:3], ctx, gamma)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.LnFp8Error):
        L.layernorm_fwd(x, gamma, beta, eps=-1.0)
    wide = torch.zeros(1, 16392, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(L.LnFp8Error):
        L.layernorm_fwd(wide, wide[0], wide[0])
    g = L.layernorm_grads(4, 64)
    g.workspace = g.workspace[:-1]
    with pytest.raises(L.LnFp8Error):
        L.layernorm_bwd(x, ctx, gamma, grads=g)
