"""The 16/32-bit operators as a training step uses them together (GPU): a pre-LN feed-forward block
LayerNorm -> FC1 + GELU -> FC2 + residual that keeps only 8-bit checkpoints, forward and backward, against the
same block in 64 bits with the same checkpoints; beside an FP8 module; captured in a graph."""
import math

import pytest

torch = pytest.importorskip("torch")
import plain64 as P  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def draw(rows, cols, seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * std + mean).to(torch.bfloat16)


def weights(D, F):
    return {"gamma": draw(1, D, 1, 0.1, 1.0)[0], "beta": draw(1, D, 2, 0.1)[0], "w1": draw(F, D, 3, 1 / math.sqrt(D)), "b1": draw(1, F, 4, 0.1)[0],
            "w2": draw(D, F, 5, 1 / math.sqrt(F)), "b2": draw(1, D, 6, 0.1)[0]}


def forward(L, x, p):
    ln, c0 = L.layernorm_fwd(x, p["gamma"], p["beta"], ckpt=True)
    a, c1 = L.linear_act_fwd(ln, p["w1"], p["b1"], act="gelu", save="ckpt")
    y, _ = L.linear_act_fwd(a, p["w2"], p["b2"], residual=x)
    return y, c0, c1


def backward(L, dy, c0, c1, p):
    g2 = L.linear_act_bwd(dy, c1.ckpt, p["w2"], L.LinearActCtx(), x_act="gelu")
    g1 = L.linear_act_bwd(g2.dx, c0.ckpt, p["w1"], c1, x_gamma=p["gamma"], x_beta=p["beta"])
    g0 = L.layernorm_bwd(g1.dx, c0, p["gamma"], dresidual=dy)
    return {"dx": g0.dx, "dgamma": g0.dgamma, "dbeta": g0.dbeta, "dw1": g1.dw, "db1": g1.dbias, "dw2": g2.dw, "db2": g2.dbias}


@pytest.mark.parametrize("M,D,F", [(1, 256, 1024), (200, 256, 512), (1030, 768, 1536)])
def test_block_against_64_bits(L, M, D, F):
    """Each 16-bit rounding on the way is half a step, 2^-9 of its tensor in the 2-norm on average; the longest way
    (dx: dA, dz1, dLN, dx and their operands) has 8, which add in quadrature below 2^-8 * sqrt(8) at worst."""
    p = weights(D, F)
    x, dy = draw(M, D, 7), draw(M, D, 8, 0.1)
    y, c0, c1 = forward(L, x, p)
    g = backward(L, dy, c0, c1, p)
    q = {k: v.double() for k, v in p.items()}
    v, d = x.double(), dy.double()
    mu = v.mean(1, keepdim=True)
    rs = ((v - mu).square().mean(1, keepdim=True) + 1e-5) ** -0.5
    h = ((v - mu) * rs * q["gamma"] + q["beta"]) @ q["w1"].t() + q["b1"]
    want_y = P.act(h, "gelu") @ q["w2"].t() + q["b2"] + v
    xh, hq = P.decode(c0.ckpt.codes, c0.ckpt.scales, 0), P.decode(c1.ckpt.codes, c1.ckpt.scales, 0)
    dz1 = (d @ q["w2"]) * P.slope(hq, "gelu")
    dln = dz1 @ q["w1"]
    gg = dln * q["gamma"]
    want = {"dx": rs * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True)) + d, "dgamma": (dln * xh).sum(0),
            "dbeta": dln.sum(0), "dw1": dz1.t() @ (xh * q["gamma"] + q["beta"]), "db1": dz1.sum(0), "dw2": d.t() @ P.act(hq, "gelu"),
            "db2": d.sum(0)}
    tol = 2.0 ** -8 * math.sqrt(8)
    assert float((y.double() - want_y).norm() / want_y.norm()) < tol
    for k, t in want.items():
        assert float((g[k].double() - t).norm() / t.norm()) < tol, k
    L.sync_status()


def test_gradients_close_to_those_without_checkpoints(L):
    """What the 8 bits cost: codes are off by at most 2^-4 of a value, 2^-4 / sqrt(3) on average, so gradients that
    are sums of products with them stay within 2^-4 of those computed from the tensors themselves."""
    M, D, F = 512, 256, 1024
    p = weights(D, F)
    x, dy = draw(M, D, 7), draw(M, D, 8, 0.1)
    y, c0, c1 = forward(L, x, p)
    g = backward(L, dy, c0, c1, p)
    ln, k0 = L.layernorm_fwd(x, p["gamma"], p["beta"])
    a, k1 = L.linear_act_fwd(ln, p["w1"], p["b1"], act="gelu", save="h")
    g2 = L.linear_act_bwd(dy, a, p["w2"], L.LinearActCtx())
    g1 = L.linear_act_bwd(g2.dx, ln, p["w1"], k1)
    g0 = L.layernorm_bwd(g1.dx, k0, p["gamma"], dresidual=dy)
    for k, t in {"dx": g0.dx, "dgamma": g0.dgamma, "dw1": g1.dw, "dw2": g2.dw, "db1": g1.dbias}.items():
        assert float((g[k].double() - t.double()).norm() / t.double().norm()) < 2.0 ** -4, k


def test_block_in_a_graph_beside_an_fp8_module(L):
    M, D, F = 256, 256, 512
    p = weights(D, F)
    x, dy = draw(M, D, 7), draw(M, D, 8, 0.1)
    rec, meta = L.Recipe("hybrid", 4), L.ScalingMeta(4, 4)

    def step():
        y, c0, c1 = forward(L, x, p)
        z, _ = L.ln_mlp_fwd(y, p["gamma"], p["beta"], p["w1"], p["b1"], p["w2"], p["b2"], meta, rec, defer_update=True)
        return [y, z] + list(backward(L, dy, c0, c1, p).values())

    step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    x.copy_(draw(M, D, 17))
    gr.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    L.sync_status()


def test_two_streams_at_once(L):
    """Two blocks in flight on two streams, each with its own workspaces, give what one at a time gives."""
    p = weights(256, 512)
    xs, dys = [draw(900, 256, 70 + i) for i in range(2)], [draw(900, 256, 80 + i, 0.1) for i in range(2)]

    def whole(i):
        y, c0, c1 = forward(L, xs[i], p)
        return [y] + list(backward(L, dys[i], c0, c1, p).values())

    want = [whole(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = whole(i)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_gradients_keep_no_scratch(L):
    """What the backward calls return holds the gradients and nothing else; handed back, they are filled again (a
    training loop's static buffers), with a workspace of the caller's or one of the call's own: the same bits."""
    M, D, F = 1030, 256, 1024
    p = weights(D, F)
    x, dy = draw(M, D, 7), draw(M, D, 8, 0.1)
    _, c0, c1 = forward(L, x, p)
    da = draw(M, F, 9, 0.1)
    calls = {
        "linear_act": lambda grads=None: L.linear_act_bwd(da, c0.ckpt, p["w1"], c1, x_gamma=p["gamma"], x_beta=p["beta"], grads=grads),
        "layernorm": lambda grads=None: L.layernorm_bwd(dy, c0, p["gamma"], dresidual=dy, grads=grads),
    }
    own = {"linear_act": L.linear_act_grads(M, D, F, act="gelu", x_from_ckpt=True), "layernorm": L.layernorm_grads(M, D)}

    def check(name, call):
        call()
        torch.cuda.synchronize()
        held = "requested_bytes.all.current"
        before = torch.cuda.memory_stats()[held]
        g = call()
        fields = {k: v for k, v in vars(g).items() if v is not None}
        assert "workspace" not in fields
        assert torch.cuda.memory_stats()[held] - before == sum(v.nbytes for v in fields.values()), name
        want = {k: v.clone() for k, v in fields.items()}
        for again in (call(g), call(own[name])):
            for k, v in want.items():
                assert torch.equal(getattr(again, k), v), (name, k)
                getattr(again, k).zero_()
        assert g.workspace is None and own[name].workspace is not None

    for name, call in calls.items():
        check(name, call)
