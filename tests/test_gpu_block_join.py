"""block_join_fwd / block_join_bwd (GPU) against the formulas in 64 bits. A row's sum is at most 16 terms one after another in
a thread and a tree of ten steps above them, so its error is at most 32 U of the terms' magnitudes (U = 2^-24); a square root and
a division of the statistics are within 4 U. Errors of intermediate values are carried along to the outputs' own rounding."""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")
import draws64 as D  # noqa: E402
import plain64 as P  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# rows, columns: one row, one column, the borders between the row shapes, odd and unaligned widths, the widest
SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 64), (70, 128), (33, 250), (40, 256), (9, 457), (17, 512), (700, 768), (6, 1000), (11, 1001), (300, 1024), (5, 2040),
          (513, 2048), (7, 2056), (5, 4096), (4, 4104), (3, 8192), (4, 8200), (3, 16383), (2, 16384)]
EPS = 1e-5
U = P.U
S = 32 * U


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def draw(rows, cols, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * std + mean).to(dtype)


def vectors(cols, names, dtype, seed=50):
    kinds = {"post_gamma": (0.1, 1.0), "post_beta": (0.1, 0.0), "gate": (0.3, 0.5), "pre_gamma": (0.1, 1.0), "pre_beta": (0.1, 0.0)}
    return {n: draw(1, cols, dtype, seed + i, *kinds[n])[0] for i, n in enumerate(kinds) if n in names}


def normed(v, ev, layer):
    """Normalised rows, rsigma and mean of v known to ev, and the first two's error bounds."""
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    mu = mean(v) if layer else torch.zeros_like(v[:, :1])
    emu = mean(ev) + S * mean(v.abs()) if layer else 0.0 * mu
    dev = v - mu
    edev = ev + emu + U * dev.abs()
    var = mean(dev * dev) + EPS
    evar = mean(2 * dev.abs() * edev + edev * edev) + (S + 2 * U) * var
    rs = var ** -0.5
    # of 1 / sqrt between var - evar and var + evar
    ers = ((var - evar).clamp_min(EPS * (1 - 4 * U)) ** -0.5 - rs).clamp_min(0) + (0.5 * evar / var + 4 * U) * rs
    return dev * rs, rs, mu, edev * (rs + ers) + dev.abs() * ers + U * (dev * rs).abs(), ers, emu


def back(g, eg, xh, exh, rs, layer):
    """rs (g - [mean g] - xh mean(g xh)) and its error bound."""
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    m1, m2 = mean(g), mean(g * xh)
    e1 = mean(eg) + (S + U) * mean(g.abs())
    e2 = mean(eg * (xh.abs() + exh) + g.abs() * exh) + (S + 2 * U) * mean((g * xh).abs())
    if not layer:
        m1, e1 = 0 * m1, 0 * e1
    out = rs * (g - m1 - xh * m2)
    mag = g.abs() + m1.abs() + (xh * m2).abs()
    return out, rs * (eg + e1 + xh.abs() * e2 + exh * (m2.abs() + e2) + 4 * U * mag)


def rounded(want, tol, dtype):
    return tol + (P.half(dtype) * (want.abs() + tol) + P.tiny(dtype) if dtype != torch.float32 else U * (want.abs() + tol) + 1e-44)


def keep_of(shape, p, seed, step, site):
    if D.cut_of(p) == 0:
        return torch.ones(shape, dtype=torch.float64, device="cuda")
    return D.keep(*shape, p, seed, step, site).cuda().double() * D.factor(p)


def check_fwd(h, y, ctx, x, r, vec, norm, scale, keep, row_stats=True):
    dt, layer = x.dtype, norm == "layer"
    v = {k: t.double() for k, t in vec.items()}
    n, en = x.double(), torch.zeros_like(x, dtype=torch.float64)
    if "post_gamma" in v:
        n, rs, mu, en, ers, emu = normed(n, en, layer)
        P.assert_within(ctx.post_rsigma[:, None], rs, ers + U * rs, "post_rsigma")
        if layer:
            P.assert_within(ctx.post_mu[:, None], mu, emu + U * mu.abs(), "post_mu")
        b = v.get("post_beta", 0.0 * v["post_gamma"])
        mag = (n * v["post_gamma"]).abs() + b.abs()
        n, en = n * v["post_gamma"] + b, en * v["post_gamma"].abs() + 4 * U * mag
    f = scale * keep * v.get("gate", 1.0)
    t, et = n * f, (en + 4 * U * n.abs()) * f.abs()
    if "post_beta" in v:
        et = et + 4 * U * mag * f.abs()
    want = t + (r.double() if r is not None else 0.0)
    P.assert_within(h, want, rounded(want, et + U * want.abs(), dt), "h")
    if "pre_gamma" not in v:
        assert y is None
        return
    hh, rs, mu, ehh, ers, emu = normed(h.double(), torch.zeros_like(want), layer)
    P.assert_within(ctx.pre_rsigma[:, None], rs, ers + U * rs, "pre_rsigma")
    if layer:
        P.assert_within(ctx.pre_mu[:, None], mu, emu + U * mu.abs(), "pre_mu")
    b = v.get("pre_beta", 0.0 * v["pre_gamma"])
    want = hh * v["pre_gamma"] + b
    P.assert_within(y, want, rounded(want, ehh * v["pre_gamma"].abs() + 2 * U * ((hh * v["pre_gamma"]).abs() + b.abs()), dt), "y")


def check_bwd(g, dh, dy, ctx, vec, keep):
    layer, scale = ctx.norm == "layer", ctx.scale
    one = dh if dh is not None else dy
    dt, M = one.dtype, one.shape[0]
    v = {k: t.double() for k, t in vec.items()}
    n_sum = (M / 152 + 60) * U  # rows of a thread, row groups, the blocks' partial sums and their lanes

    def given(part, t):
        rs = getattr(ctx, part + "_rsigma")[:, None].double()
        mu = getattr(ctx, part + "_mu")[:, None].double() if layer else 0.0
        xh = (t.double() - mu) * rs
        return xh, 3 * U * xh.abs(), rs

    def column(name, t, et):
        P.assert_within(getattr(g, name), t.sum(0), et.sum(0) + n_sum * t.abs().sum(0) + 1e-44, name)

    d = dh.double() if dh is not None else torch.zeros_like(one, dtype=torch.float64)
    ed = torch.zeros_like(d)
    if "pre_gamma" in v:
        hh, ehh, rs = given("pre", ctx.h)
        q = dy.double() * v["pre_gamma"]
        o, eo = back(q, U * q.abs(), hh, ehh, rs, layer)
        column("dpre_gamma", dy.double() * hh, dy.double().abs() * ehh)
        if "pre_beta" in v:
            column("dpre_beta", dy.double(), ed)
        d, ed = d + o, eo + U * (d.abs() + o.abs())
    if g.dresidual is not None:
        P.assert_within(g.dresidual, d, rounded(d, ed, dt), "dresidual")
    f = scale * keep
    t, et = d * f, ed * f.abs() + 3 * U * (d * f).abs()
    gate = v.get("gate", torch.ones_like(one[0], dtype=torch.float64))
    if "post_gamma" in v:
        xh, exh, rs = given("post", ctx.x)
        bare, n, en = xh, xh * v["post_gamma"] + v.get("post_beta", 0.0), exh * v["post_gamma"].abs()
        column("dpost_gamma", t * gate * xh, gate.abs() * (et * (xh.abs() + exh) + t.abs() * exh) + 2 * U * (t * gate * xh).abs())
        if "post_beta" in v:
            column("dpost_beta", t * gate, et * gate.abs() + 2 * U * (t * gate).abs())
    elif "gate" in v:
        n, en = ctx.x.double(), torch.zeros_like(d)
    if "gate" in v:
        if "post_beta" in v:  # two sums are added
            pieces = ((t * xh * v["post_gamma"]).abs() + (t * v["post_beta"]).abs()).sum(0)
            P.assert_within(g.dgate, (t * n).sum(0), (et * (n.abs() + en) + t.abs() * en).sum(0) + (et * v["post_beta"].abs()).sum(0) + (n_sum + 4 * U) * pieces + 1e-44, "dgate")
        else:
            column("dgate", t * n, et * (n.abs() + en) + t.abs() * en + 2 * U * (t * n).abs())
    u, eu = t * gate, et * gate.abs() + U * (t * gate).abs()
    if "post_gamma" in v:
        u, eu = u * v["post_gamma"], eu * v["post_gamma"].abs() + 2 * U * (u * v["post_gamma"]).abs()
        u, eu = back(u, eu, xh, exh, rs, layer)
    P.assert_within(g.dx, u, rounded(u, eu, dt), "dx")


ALL = ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta")
SETS = {"full": ALL, "rms_block": ("post_gamma", "pre_gamma"), "gate_pre": ("gate", "pre_gamma", "pre_beta"), "post_only": ("post_gamma", "post_beta"),
        "plain": (), "gate_post": ("post_gamma", "gate"), "pre_only": ("pre_gamma",)}


def run_both(L, M, C, dtype, norm, names, p, scale, pdtype=None, residual=True, strided=False, with_dh=True, seed=3):
    def tensor(s, std=1.0):
        return draw(M, C + (24 if strided else 0), dtype, s, std)[:, (5 if strided else 0) :][:, :C]
    x, r = tensor(1, 2.0), tensor(2, 3.0) if residual else None
    vec = vectors(C, names, pdtype or dtype)
    rng = L.dropout_rng(seed, step=4)
    h, y, ctx = L.block_join_fwd(x, r, norm=norm, scale=scale, p=p, rng=rng, site=6, eps=EPS, **vec)
    keep = keep_of((M, C), p, seed, 4, 6)
    check_fwd(h, y, ctx, x, r, vec, norm, scale, keep)
    dh, dy = tensor(3, 0.1) if with_dh or "pre_gamma" not in names else None, tensor(4, 0.1) if "pre_gamma" in names else None
    rng += 5
    g = L.block_join_bwd(dh, dy, ctx, **vec)
    check_bwd(g, dh, dy, ctx, vec, keep)
    again = L.block_join_bwd(dh, dy, ctx, **vec)
    for k in ("dx", "dresidual", "dpost_gamma", "dpost_beta", "dgate", "dpre_gamma", "dpre_beta"):
        a, b = getattr(g, k), getattr(again, k)
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b)), k
        want = k[1:] in names or k in ("dx", "dresidual")
        assert (a is not None) == want, k


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", SHAPES)
@pytest.mark.parametrize("norm,names,p", [("rms", "rms_block", 0.1), ("layer", "full", 0.3), ("layer", "gate_pre", 0.0)])
def test_shapes(L, M, C, dtype, norm, names, p):
    run_both(L, M, C, dtype, norm, SETS[names], p, 0.5 if names == "full" else 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("C", [250, 1001, 4104, 8200, 12000, 16384])
@pytest.mark.parametrize("norm,names,p", [("rms", "rms_block", 0.1), ("layer", "full", 0.0), ("rms", "gate_post", 0.2)])
def test_several_rows_to_a_block(L, C, dtype, norm, names, p):
    run_both(L, 470, C, dtype, norm, SETS[names], p, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [264, 512, 776, 1024, 1544, 2048, 3080, 4096, 6152, 7168, 8192])
@pytest.mark.parametrize("norm,names,p", [("rms", "rms_block", 0.1), ("layer", "full", 0.0), ("layer", "full", 0.1), ("layer", "gate_pre", 0.0)])
def test_columns_a_thread(L, C, dtype, norm, names, p):
    """Both borders of the widths with 32 columns a thread where a row is much work, and parts with which it is not."""
    run_both(L, 701, C, dtype, norm, SETS[names], p, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [520, 640, 776, 1032, 1280, 2056, 2560, 3064, 4104, 5120, 6136, 6152])
@pytest.mark.parametrize("norm,names,p", [("rms", "rms_block", 0.1), ("layer", "full", 0.0), ("layer", "gate_pre", 0.2)])
def test_rows_shared_by_threads_that_are_no_power_of_two(L, C, dtype, norm, names, p):
    """Both borders of the widths between powers of two, several rows to a group of threads and one group without any."""
    run_both(L, 701, C, dtype, norm, SETS[names], p, 1.0)


@pytest.mark.parametrize("C", [96, 1001, 2048, 8200])
@pytest.mark.parametrize("names", list(SETS))
@pytest.mark.parametrize("norm,p,residual", list(itertools.product(("rms", "layer"), (0.0, 0.2), (True, False))))
def test_every_set_of_parts(L, C, names, norm, p, residual):
    run_both(L, 37, C, torch.bfloat16, norm, SETS[names], p, 0.22, residual=residual, with_dh=residual)


@pytest.mark.parametrize("dtype,pdtype", list(itertools.product(DTYPES, DTYPES)))
@pytest.mark.parametrize("C", [264, 1003])
def test_types_of_the_vectors(L, dtype, pdtype, C):
    run_both(L, 20, C, dtype, "layer", ALL, 0.1, 1.0, pdtype=pdtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [48, 768, 8192])
def test_strided_unaligned_rows(L, C, dtype):
    """Rows that start at an odd element: the kernels of any alignment at widths that the others take otherwise."""
    run_both(L, 21, C, dtype, "rms", ("post_gamma", "gate", "pre_gamma"), 0.25, 1.0, strided=True)


@pytest.mark.parametrize("C", [64, 2048, 8200, 12000])
def test_vectors_on_odd_boundaries(L, C):
    """Rows on 16-byte boundaries, vectors that start at any element."""
    M, dt = 9, torch.bfloat16
    x, r, dh, dy = (draw(M, C, dt, s) for s in (1, 2, 3, 4))
    vec = {k: torch.cat((v[:3], v))[3:] for k, v in vectors(C, ALL, dt).items()}
    assert all(v.data_ptr() % 16 for v in vec.values())
    h, y, ctx = L.block_join_fwd(x, r, norm="layer", **vec)
    keep = keep_of((M, C), 0.0, 0, 0, 0)
    check_fwd(h, y, ctx, x, r, vec, "layer", 1.0, keep)
    check_bwd(L.block_join_bwd(dh, dy, ctx, **vec), dh, dy, ctx, vec, keep)


@pytest.mark.parametrize("C", [2048, 1001])
def test_given_buffers_and_what_lies_around_them(L, C):
    M, dt = 45, torch.bfloat16
    x, r, vec = draw(M, C, dt, 1), draw(M, C, dt, 2), vectors(C, ALL, dt)
    big = lambda: torch.full((M + 3, C + 40), 7.0, dtype=dt, device="cuda")  # noqa: E731
    hb, yb, xb, rb = big(), big(), big(), big()
    part = lambda t: t[:M, 16 : 16 + C]  # noqa: E731
    h, y, ctx = L.block_join_fwd(x, r, norm="layer", h=part(hb), y=part(yb), **vec)
    check_fwd(h, y, ctx, x, r, vec, "layer", 1.0, keep_of((M, C), 0.0, 0, 0, 0))
    g = L.block_join_grads(M, C, post_gamma=True, post_beta=True, gate=True, pre_gamma=True, pre_beta=True)
    g.dx, g.dresidual = part(xb), part(rb)
    dh, dy = draw(M, C, dt, 3), draw(M, C, dt, 4)
    L.block_join_bwd(dh, dy, ctx, grads=g, **vec)
    check_bwd(g, dh, dy, ctx, vec, keep_of((M, C), 0.0, 0, 0, 0))
    for t in (hb, yb, xb, rb):
        part(t).fill_(7.0)
        assert (t == 7.0).all()
    g2 = L.block_join_grads(M, C, dresidual=False, post_gamma=True, post_beta=True, gate=True, pre_gamma=True, pre_beta=True)
    L.block_join_bwd(dh, dy, ctx, grads=g2, **vec)
    assert g2.dresidual is None
    check_bwd(g2, dh, dy, ctx, vec, keep_of((M, C), 0.0, 0, 0, 0))


@pytest.mark.parametrize("C", [512, 515])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_rows_far_from_zero(L, C, norm):
    """A mean a thousand deviations from zero, a constant row, a row of zeros."""
    x = draw(6, C, torch.float32, 1, 1.0, 1000.0)
    x[2], x[3] = 5.0, 0.0
    vec = vectors(C, ALL, torch.float32)
    h, y, ctx = L.block_join_fwd(x, None, norm=norm, eps=EPS, **vec)
    check_fwd(h, y, ctx, x, None, vec, norm, 1.0, keep_of((6, C), 0.0, 0, 0, 0))


@pytest.mark.parametrize("C", [64, 2048, 1001])
def test_nan_stays_in_its_row_and_dropped_elements_count_for_nothing(L, C):
    M, dt, p = 40, torch.bfloat16, 0.5
    x, r = draw(M, C, dt, 1), draw(M, C, dt, 2)
    x[3, C // 2], x[7, 0] = math.nan, math.inf
    rng = L.dropout_rng(2)
    k = D.keep(M, C, p, 2, 0, 0).cuda()
    vec = vectors(C, ("pre_gamma",), dt)
    h, y, ctx = L.block_join_fwd(x, r, p=p, rng=rng, **vec)
    assert torch.equal(h.isfinite(), x.isfinite() | ~k) and torch.equal(h[~k], r[~k])
    bad = ~h.isfinite().all(1)
    assert y[~bad].isfinite().all()
    vec = vectors(C, ("post_gamma", "pre_gamma"), dt)
    h, y, ctx = L.block_join_fwd(x, r, p=p, rng=rng, **vec)
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[3] = rows[7] = False
    assert h[rows].isfinite().all() and y[rows].isfinite().all() and h[3][k[3]].isnan().all() and torch.equal(h[3][~k[3]], r[3][~k[3]])
    dh = draw(M, C, dt, 5)
    dh[11, C // 3] = math.nan
    ctx2 = L.block_join_fwd(r, r, p=p, rng=rng, **vec)[2]
    g = L.block_join_bwd(dh, draw(M, C, dt, 6), ctx2, **vec)
    rows[:] = True
    rows[11] = False
    assert g.dx[rows].isfinite().all() and g.dresidual[rows].isfinite().all() and g.dresidual[11].isnan().sum() == 1
    assert g.dx[11].isnan().all() == bool(k[11, C // 3])


def test_no_rows(L):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    vec = vectors(64, ALL, torch.bfloat16)
    h, y, ctx = L.block_join_fwd(x, x, **vec)
    g = L.block_join_bwd(h, y, ctx, **vec)
    assert h.shape == y.shape == g.dx.shape == (0, 64)
    for n in ALL:
        assert (getattr(g, "d" + n) == 0).all()


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("C", [40, 129])
def test_gradients_agree_with_differences(L, norm, C):
    """In fp32, the loss sum(c h) + sum(e y) along a random direction of each input: a central difference with step 2^-7 is the
    slope up to the third derivative and 2^7 U of the loss's terms."""
    M = 12
    x, r, c, e = (draw(M, C, torch.float32, s) for s in (1, 2, 3, 4))
    vec = vectors(C, ALL, torch.float32)
    kw = dict(norm=norm, scale=0.7, p=0.3, rng=L.dropout_rng(8), site=1)

    def loss(x, r, vec):
        h, y, ctx = L.block_join_fwd(x, r, **kw, **vec)
        return float((c.double() * h.double()).sum() + (e.double() * y.double()).sum()), ctx, float((c * h).abs().sum() + (e * y).abs().sum())

    _, ctx, size = loss(x, r, vec)
    g = L.block_join_bwd(c, e, ctx, **vec)
    grads = {"x": g.dx, "r": g.dresidual, **{n: getattr(g, "d" + n) for n in ALL}}
    step = 2.0 ** -7
    for i, (name, grad) in enumerate(grads.items()):
        v = draw(*(grad.shape if grad.dim() == 2 else (1, C)), torch.float32, 20 + i).reshape(grad.shape)
        f = []
        for s in (step, -step):
            xs, rs, vs = x, r, dict(vec)
            if name == "x":
                xs = x + s * v
            elif name == "r":
                rs = r + s * v
            else:
                vs[name] = vec[name] + s * v
            f.append(loss(xs, rs, vs)[0])
        slope = float((grad.double() * v.double()).sum())
        scale = float((grad.double() * v.double()).abs().sum())
        assert abs((f[0] - f[1]) / (2 * step) - slope) < 4 * step ** 2 * scale + 64 * U / step * size, name


@pytest.mark.parametrize("M,C", [(1, 2048), (300, 768), (50, 1001)])
def test_other_stream_and_graph(L, M, C):
    dt = torch.bfloat16
    x, r, dh, dy = (draw(M, C, dt, s) for s in (1, 2, 3, 4))
    vec = vectors(C, ALL, dt)
    rng = L.dropout_rng(5)
    torch.cuda.synchronize()

    def step(stream=None):
        h, y, ctx = L.block_join_fwd(x, r, p=0.2, rng=rng, **vec, stream=stream)
        g = L.block_join_bwd(dh, dy, ctx, **vec, stream=stream)
        return [h, y, g.dx, g.dresidual] + [getattr(g, "d" + n) for n in ALL]

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    rng[1] += 1
    x.copy_(draw(M, C, dt, 9))
    want = step()
    for gr, out in graphs + graphs:
        gr.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("C", [8192, 1001])
def test_offsets_past_32_bits(L, C):
    M, dt = (1 << 31) // C + 70, torch.bfloat16
    x = draw(64, C, dt, 1).repeat(M // 64 + 1, 1)[:M]
    vec = vectors(C, ("post_gamma", "pre_gamma"), dt)
    rng = L.dropout_rng(5)
    h, y, ctx = L.block_join_fwd(x, x, p=0.1, rng=rng, **vec)
    g = L.block_join_bwd(y, h, ctx, **vec)
    for lo in (0, M - 40):
        part = slice(lo, lo + 40)
        keep = D.keep(40, C, 0.1, 5, 0, 0, row0=lo).cuda().double() * D.factor(0.1)
        c2 = L.BlockJoinCtx(x[part], h[part], "rms", 1.0, 0.1, None, 0, None, ctx.post_rsigma[part], None, ctx.pre_rsigma[part])
        check_fwd(h[part], y[part], c2, x[part], x[part], vec, "rms", 1.0, keep)

        class Part:  # of the gradients, without the column sums of all rows
            dx, dresidual = g.dx[part], g.dresidual[part]
        few = L.BlockJoinGrads(Part.dx, Part.dresidual)
        check_rows(few, y[part], h[part], c2, vec, keep)


def check_rows(g, dh, dy, ctx, vec, keep):
    """check_bwd without the column sums: a stand-in takes their place."""
    class Any:
        dx, dresidual = g.dx, g.dresidual

        def __getattr__(self, name):
            return None
    within = P.assert_within
    try:
        P.assert_within = lambda got, want, tol, what: within(got, want, tol, what) if got is not None else None
        check_bwd(Any(), dh, dy, ctx, vec, keep)
    finally:
        P.assert_within = within


def test_refusals(L):
    x = draw(8, 64, torch.bfloat16, 1)
    v = vectors(64, ALL, torch.bfloat16)
    with pytest.raises(ValueError, match="needs rng"):
        L.block_join_fwd(x, x, p=0.1)
    with pytest.raises(ValueError, match="residual has shape"):
        L.block_join_fwd(x, x[:7])
    with pytest.raises(TypeError, match="pre_gamma is"):
        L.block_join_fwd(x, x, gate=v["gate"], pre_gamma=v["pre_gamma"].float())
    with pytest.raises(ValueError, match="y without"):
        L.block_join_fwd(x, x, y=torch.empty_like(x))
    with pytest.raises(L.LnFp8Error, match="post_beta"):
        L.block_join_fwd(x, x, post_beta=v["post_beta"])
    with pytest.raises(L.LnFp8Error, match="eps"):
        L.block_join_fwd(x, x, eps=-1.0)
    h, y, ctx = L.block_join_fwd(x, x, pre_gamma=v["pre_gamma"])
    with pytest.raises(ValueError, match="statistics"):
        L.block_join_bwd(x, x, ctx, post_gamma=v["post_gamma"], pre_gamma=v["pre_gamma"])
    with pytest.raises(ValueError, match="ctx.x is missing"):
        L.block_join_bwd(x, x, ctx, gate=v["gate"], pre_gamma=v["pre_gamma"])
    with pytest.raises(L.LnFp8Error, match="dy"):
        L.block_join_bwd(x, None, ctx, pre_gamma=v["pre_gamma"])
    with pytest.raises(L.LnFp8Error, match="dy without"):
        L.block_join_bwd(x, x, ctx)
    with pytest.raises(ValueError, match="pre_beta without"):
        L.block_join_bwd(x, None, ctx, pre_beta=v["pre_beta"])
    g = L.block_join_grads(8, 64, pre_gamma=True)
    g.workspace = g.workspace[:16]
    with pytest.raises(L.LnFp8Error, match="workspace"):
        L.block_join_bwd(x, x, ctx, pre_gamma=v["pre_gamma"], grads=g)
