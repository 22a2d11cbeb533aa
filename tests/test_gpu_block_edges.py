"""block_join and dropout where they can go wrong at the edges (GPU). Bounds as in test_gpu_block_join.py."""
import math

import pytest

torch = pytest.importorskip("torch")
import draws64 as D  # noqa: E402
import plain64 as P  # noqa: E402
from test_gpu_block_join import ALL, DTYPES, EPS, U, back, check_bwd, draw, keep_of, normed, rounded, vectors  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


ROWS_DROPPED = [pytest.param(dt, C, norm, names, id=f"{str(dt)[6:]}-{C}-{norm}") for dt in DTYPES for C in (1, 7, 8, 24, 40)
                for norm, names in (("rms", ("post_gamma", "pre_gamma")), ("layer", ALL))]


def dropped_rows(M, C, p, seed):
    none = ~D.keep(M, C, p, seed, 0, 0).any(1).cuda()
    assert 4 <= int(none.sum()) < M
    return none


@pytest.mark.parametrize("dtype,C,norm,names", ROWS_DROPPED)
def test_a_row_whose_elements_are_all_dropped_is_the_residual(L, dtype, C, norm, names):
    """x's rows are NaN throughout once normalised, and count for nothing where they are dropped."""
    M, p, layer = 600, 0.9, norm == "layer"
    x, r = draw(M, C, dtype, 1), draw(M, C, dtype, 2)
    x[:, C // 2] = math.nan
    vec, none = vectors(C, names, dtype), dropped_rows(M, C, p, 13)
    h, y, ctx = L.block_join_fwd(x, r, norm=norm, p=p, rng=L.dropout_rng(13), eps=EPS, **vec)
    assert torch.equal(h[none], r[none]) and h[~none].isnan().any(1).all() and y[~none].isnan().all()
    hh, rs, mu, ehh, ers, emu = normed(h[none].double(), torch.zeros_like(h[none], dtype=torch.float64), layer)
    P.assert_within(ctx.pre_rsigma[none][:, None], rs, ers + U * rs, "pre_rsigma")
    if layer:
        P.assert_within(ctx.pre_mu[none][:, None], mu, emu + U * mu.abs(), "pre_mu")
    g2, b2 = vec["pre_gamma"].double(), vec.get("pre_beta", 0 * vec["pre_gamma"]).double()
    want = hh * g2 + b2
    P.assert_within(y[none], want, rounded(want, ehh * g2.abs() + 2 * U * ((hh * g2).abs() + b2.abs()), dtype), "y")


@pytest.mark.parametrize("dtype,C,norm,names", ROWS_DROPPED)
def test_a_row_whose_elements_are_all_dropped_has_no_gradient(L, dtype, C, norm, names):
    """The gradient of h is NaN throughout, and dx of a row that is dropped is exactly zero."""
    M, p = 600, 0.9
    x, r, dh, dy = (draw(M, C, dtype, s) for s in (1, 2, 3, 4))
    vec, none = vectors(C, names, dtype), dropped_rows(M, C, p, 13)
    ctx = L.block_join_fwd(x, r, norm=norm, p=p, rng=L.dropout_rng(13), eps=EPS, **vec)[2]
    dy[:, C // 2] = math.nan
    g = L.block_join_bwd(dh, dy, ctx, **vec)
    assert g.dresidual.isnan().all()
    assert (g.dx[none] == 0).all() and g.dx[~none].isnan().all()


@pytest.mark.parametrize("dtype,C", [(torch.bfloat16, 64), (torch.float16, 65), (torch.bfloat16, 8200), (torch.bfloat16, 8201),
                                     (torch.float32, 64), (torch.float32, 65), (torch.float32, 8196)])
@pytest.mark.parametrize("post", [False, True])
def test_an_infinite_gate_without_a_beta(L, dtype, C, post):
    """gate x is infinite in that column with the sign of x, and nothing else of h changes."""
    M, at = 20, C // 2
    x, r = draw(M, C, dtype, 1), draw(M, C, dtype, 2)
    x[:, at] = torch.where(torch.arange(M, device="cuda") % 2 == 0, 2.0, -3.0).to(dtype)
    vec = vectors(C, ("gate", "pre_gamma", "pre_beta") + (("post_gamma",) if post else ()), dtype)
    vec["gate"][at] = 1.0
    want = L.block_join_fwd(x, r, norm="layer", **vec)[0]
    vec["gate"][at] = math.inf
    h = L.block_join_fwd(x, r, norm="layer", **vec)[0]
    assert torch.equal(h[:, at], torch.where(x[:, at] > 0, math.inf, -math.inf).to(dtype))
    assert torch.equal(h[:, :at], want[:, :at]) and torch.equal(h[:, at + 1 :], want[:, at + 1 :])


@pytest.mark.parametrize("captured", [False, True])
def test_calls_without_rows_keep_a_copy_of_rng(L, captured):
    """The context's copy is what the call read, whatever its memory held before."""
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    rng = L.dropout_rng(1234, step=5)

    def calls():
        junk = [torch.full((2,), -7, dtype=torch.int64, device="cuda") for _ in range(8)]
        del junk
        return L.dropout_fwd(x, 0.5, rng)[1].rng, L.block_join_fwd(x, x, p=0.5, rng=rng)[2].rng

    if not captured:
        got = calls()
    else:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls()
        rng[1] += 1
        graph.replay()
    assert all(torch.equal(g, rng) for g in got)


def test_a_backward_call_takes_the_vectors_of_its_forward(L):
    """What would give another operator's gradients is refused; a beta's own gradient may be left out where no other needs it, and so
    may y's part. A context made by hand that does not say which vectors there were is taken as it is."""
    M, C, dt = 6, 64, torch.bfloat16
    x, r, dh, dy = (draw(M, C, dt, s) for s in (1, 2, 3, 4))
    v = vectors(C, ALL, dt)
    post = {k: v[k] for k in ("post_gamma", "post_beta", "gate")}
    _, _, ctx = L.block_join_fwd(x, r, norm="layer", **post)
    want = L.block_join_bwd(dh, None, ctx, **post)
    for left_out, match in (("post_gamma", "post_gamma"), ("gate", "gate"), ("post_beta", "post_beta")):
        given = {k: t for k, t in post.items() if k != left_out}
        if left_out == "post_gamma":
            del given["post_beta"]
        with pytest.raises(ValueError, match=match):
            L.block_join_bwd(dh, None, ctx, **given)
    by_hand = L.BlockJoinCtx(x, None, "layer", 1.0, 0.0, None, 0, ctx.post_mu, ctx.post_rsigma)
    got = L.block_join_bwd(dh, None, by_hand, **post)
    assert torch.equal(got.dx, want.dx) and torch.equal(got.dgate, want.dgate)
    _, _, ctx = L.block_join_fwd(x, r, post_gamma=v["post_gamma"])
    with pytest.raises(ValueError, match="gate"):
        L.block_join_bwd(dh, None, ctx, post_gamma=v["post_gamma"], gate=v["gate"])
    _, _, ctx = L.block_join_fwd(x, r, post_gamma=v["post_gamma"], gate=v["gate"])
    with pytest.raises(ValueError, match="post_beta"):
        L.block_join_bwd(dh, None, ctx, **post)
    _, _, ctx = L.block_join_fwd(x, r, post_gamma=v["post_gamma"], post_beta=v["post_beta"], pre_gamma=v["pre_gamma"], pre_beta=v["pre_beta"])
    g = L.block_join_bwd(dh, dy, ctx, post_gamma=v["post_gamma"], pre_gamma=v["pre_gamma"])
    assert g.dpost_beta is None and g.dpre_beta is None and g.dpost_gamma is not None
    g = L.block_join_bwd(dh, None, ctx, post_gamma=v["post_gamma"])
    assert g.dpre_gamma is None and torch.equal(g.dresidual, dh)


@pytest.mark.parametrize("dtype,C", [(torch.bfloat16, 64), (torch.bfloat16, 65), (torch.bfloat16, 2048), (torch.bfloat16, 8192), (torch.float32, 768)])
@pytest.mark.parametrize("M", [1, 700])
def test_statistics_that_are_not_there_count_as_none(L, M, C, dtype):
    """The calls without means, or without one of the norms, directly behind one whose rows have means far from zero, which its kernel
    leaves in the shared memory that theirs takes over."""
    x, r, dh, dy = (draw(M, C, dtype, s, 1.0, mean) for s, mean in ((1, 20.0), (2, 30.0), (3, 0.0), (4, 0.0)))
    vec, keep = vectors(C, ALL, dtype), keep_of((M, C), 0.0, 0, 0, 0)
    before = L.block_join_fwd(x, r, norm="layer", eps=EPS, **vec)[2]
    calls = [(norm, names) for names in (ALL, ("post_gamma", "post_beta"), ("pre_gamma", "pre_beta"), ("gate", "pre_gamma", "pre_beta"), ("gate",))
             for norm in ("rms", "layer")]
    for norm, names in calls:
        some = {k: v for k, v in vec.items() if k in names}
        ctx = L.block_join_fwd(x, r, norm=norm, eps=EPS, **some)[2]
        e = dy if "pre_gamma" in names else None
        L.block_join_bwd(dh, dy, before, **vec)
        g = L.block_join_bwd(dh, e, ctx, **some)
        check_bwd(g, dh, e, ctx, some, keep)


@pytest.mark.parametrize("C,norm,names", [(8192, "rms", ("post_gamma", "pre_gamma")), (1001, "layer", ALL)])
def test_column_sums_past_32_bits(L, C, norm, names):
    """Every row's part in the column sums of more than 2^31 elements: all rows differ, the terms have one sign on average, and the
    gradients of the rows past 2^31 elements are 2^14 times the others', so that one of these rows (0.5% of the terms' magnitudes at least,
    a third of it of one sign), or a block's of the others (1 in 152), shows beside the bound (0.09% at most) if it is left out or counted
    twice."""
    M, dt, layer = (1 << 31) // C + 70, torch.bfloat16, norm == "layer"
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(M, C, dtype=dt, device="cuda").normal_(1.0, 1.0, generator=gen)
    vec = vectors(C, names, dt)
    h, e, ctx = L.block_join_fwd(x, x, norm=norm, eps=EPS, **vec)
    e.copy_(h)
    e[(1 << 31) // C :] *= 2.0 ** 14
    g = L.block_join_bwd(e, e, ctx, **vec)
    v = {k: t.double() for k, t in vec.items()}
    n_sum = (M / 152 + 60) * U
    gate, b1 = v.get("gate", torch.ones(C, dtype=torch.float64, device="cuda")), v.get("post_beta", torch.zeros(C, dtype=torch.float64, device="cuda"))
    total = {}

    def add(name, t, et, mag=None):
        part = torch.stack((t.sum(0), (et + n_sum * (t.abs() if mag is None else mag)).sum(0)))
        total[name] = total[name] + part if name in total else part

    rows = (1 << 25) // C
    for lo in range(0, M, rows):
        part = slice(lo, min(M, lo + rows))

        def given(name, t):
            rs = getattr(ctx, name + "_rsigma")[part][:, None].double()
            xh = (t[part].double() - (getattr(ctx, name + "_mu")[part][:, None].double() if layer else 0.0)) * rs
            return xh, 3 * U * xh.abs(), rs

        dy = e[part].double()
        hh, ehh, rs = given("pre", h)
        add("dpre_gamma", dy * hh, dy.abs() * ehh)
        q = dy * v["pre_gamma"]
        o, eo = back(q, U * q.abs(), hh, ehh, rs, layer)
        d, ed = dy + o, eo + U * (dy.abs() + o.abs())
        xh, exh, _ = given("post", x)
        add("dpost_gamma", d * gate * xh, gate.abs() * (ed * (xh.abs() + exh) + d.abs() * exh) + 2 * U * (d * gate * xh).abs())
        if layer:
            add("dpre_beta", dy, 0 * dy)
            add("dpost_beta", d * gate, ed * gate.abs() + 2 * U * (d * gate).abs())
            n, en = xh * v["post_gamma"] + b1, exh * v["post_gamma"].abs()
            pieces = (d * xh * v["post_gamma"]).abs() + (d * b1).abs()  # two sums are added
            add("dgate", d * n, ed * (n.abs() + en) + d.abs() * en + ed * b1.abs() + 4 * U * pieces, pieces)
    for name, (want, tol) in total.items():
        P.assert_within(getattr(g, name), want, tol, name)
    assert {"d" + n for n in names} == set(total)
