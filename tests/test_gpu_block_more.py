"""The gated linear layer, dropout and the join of a block's output as a training step uses them together (GPU): a feed-forward
block between two norms, forward and backward, against the same block in 64 bits with the same masks; beside an FP8 module and a
plain linear layer; captured in graphs that draw anew; one decoded token at a time."""
import math

import pytest

torch = pytest.importorskip("torch")
import draws64 as D  # noqa: E402
import plain64 as P  # noqa: E402

pytestmark = pytest.mark.gpu
SEED, STEP = 77, 3


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def draw(rows, cols, seed, std=1.0, mean=0.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * std + mean).to(dtype)


def weights(C, F):
    return {"g0": draw(1, C, 1, 0.1, 1.0)[0], "w1": draw(2 * F, C, 2, 1 / math.sqrt(C)), "b1": draw(1, 2 * F, 3, 0.1)[0], "w2": draw(C, F, 4, 1 / math.sqrt(F)),
            "b2": draw(1, C, 5, 0.1)[0], "gp": draw(1, C, 6, 0.1, 1.0)[0], "gate": draw(1, C, 7, 0.2, 0.5)[0], "g1": draw(1, C, 8, 0.1, 1.0)[0]}


def forward(L, x, p, rng, drop):
    h0, y0, c0 = L.block_join_fwd(x, None, pre_gamma=p["g0"])
    a, cg = L.linear_glu_fwd(y0, p["w1"], p["b1"], save="h")
    a, cd = L.dropout_fwd(a, drop, rng, site=1)
    z, cl = L.linear_act_fwd(a, p["w2"], p["b2"])
    h1, y1, c1 = L.block_join_fwd(z, h0, post_gamma=p["gp"], gate=p["gate"], scale=0.5, p=drop, rng=rng, site=2, pre_gamma=p["g1"])
    return h1, y1, (c0, cg, cd, cl, c1, y0, a)


def backward(L, dh, dy, kept, p):
    c0, cg, cd, cl, c1, y0, a = kept
    j1 = L.block_join_bwd(dh, dy, c1, post_gamma=p["gp"], gate=p["gate"], pre_gamma=p["g1"])
    l2 = L.linear_act_bwd(j1.dx, a, p["w2"], cl)
    l1 = L.linear_glu_bwd(L.dropout_bwd(l2.dx, cd), y0, p["w1"], cg)
    j0 = L.block_join_bwd(j1.dresidual, l1.dx, c0, pre_gamma=p["g0"])
    return {"x": j0.dx, "g0": j0.dpre_gamma, "w1": l1.dw, "b1": l1.dbias, "w2": l2.dw, "b2": l2.dbias, "gp": j1.dpost_gamma, "gate": j1.dgate, "g1": j1.dpre_gamma}


def plain(x, p, k1, k2):
    norm = lambda v: v * (v.square().mean(1, keepdim=True) + 1e-5) ** -0.5  # noqa: E731
    z = (norm(x) * p["g0"]) @ p["w1"].t() + p["b1"]
    F = z.shape[1] // 2
    a = P.act(z[:, :F], "silu") * z[:, F:] * k1
    h = x + 0.5 * k2 * p["gate"] * norm(a @ p["w2"].t() + p["b2"]) * p["gp"]
    return h, norm(h) * p["g1"]


@pytest.mark.parametrize("M,C,F,drop", [(1, 256, 512, 0.0), (3, 264, 200, 0.2), (200, 256, 680, 0.1), (1030, 768, 2048, 0.3)])
def test_block_against_64_bits(L, M, C, F, drop):
    """A rounding to bf16 is 2^-9 of its tensor in the 2-norm on average, 2^-8 at worst. The longest way (dx: y0, h, a, z and the
    gradients dz, da, dz1, dy0, dx) has 12 of them with their operands, which add in quadrature."""
    p = weights(C, F)
    x, dh, dy = draw(M, C, 11), draw(M, C, 12, 0.1), draw(M, C, 13, 0.1)
    rng = L.dropout_rng(SEED, step=STEP)
    h, y, kept = forward(L, x, p, rng, drop)
    rng[1] += 1  # the backward draws as the forward did
    got = backward(L, dh, dy, kept, p)
    keep = lambda cols, site: (D.keep(M, cols, drop, SEED, STEP, site).double() * D.factor(drop)).cuda()  # noqa: E731
    q = {k: v.double().requires_grad_(True) for k, v in p.items()}
    xd = x.double().requires_grad_(True)
    want_h, want_y = plain(xd, q, keep(F, 1), keep(C, 2))
    grads = torch.autograd.grad((want_h * dh.double()).sum() + (want_y * dy.double()).sum(), [xd] + list(q.values()))
    tol = 2.0 ** -8 * math.sqrt(12)
    for name, g, w in [("h", h, want_h), ("y", y, want_y)] + list(zip(["x"] + list(q), [got["x"]] + [got[k] for k in q], grads)):
        assert float((g.double() - w.detach()).norm() / w.detach().norm()) < tol, name
    L.sync_status()


def test_block_in_graphs_beside_an_fp8_module(L):
    """Two graphs of the same step, replayed in turn and with the step of the draws advanced inside: each replay equals the step
    called directly."""
    M, C, F = 256, 256, 512
    p = weights(C, F)
    x, dh, dy = draw(M, C, 11), draw(M, C, 12, 0.1), draw(M, C, 13, 0.1)
    w1, w2, b1, b2 = draw(F, C, 21, 0.05), draw(C, F, 22, 0.05), draw(1, F, 23)[0], draw(1, C, 24)[0]
    rec, meta = L.Recipe("hybrid", 4), L.ScalingMeta(4, 4)

    def step(rng):
        h, y, kept = forward(L, x, p, rng, 0.2)
        m, _ = L.ln_mlp_fwd(y, p["g1"], b2, w1, b1, w2, b2, meta, rec, defer_update=True)
        rng[1] += 1
        return [h, y, m] + list(backward(L, dh, dy, kept, p).values())

    rng = L.dropout_rng(5)
    wants = [step(rng) for _ in range(4)]
    torch.cuda.synchronize()
    assert not torch.equal(wants[0][0], wants[1][0])
    rng.copy_(L.dropout_rng(5))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(rng)
        graphs.append((g, out))
    rng.copy_(L.dropout_rng(5))
    for i, want in enumerate(wants):
        g, out = graphs[i % 2]
        g.replay()
        for a, b in zip(want, out):
            assert torch.equal(a, b)


def test_decoding_row_by_row_gives_the_batch(L):
    """A row alone and in a batch takes other kernels for its products, whose sums are in another order: within the roundings of
    the way, and bit for bit where nothing is summed over more than the row."""
    M, C, F = 40, 512, 1024
    p = weights(C, F)
    x = draw(M, C, 11)
    h, y, _ = forward(L, x, p, None, 0.0)
    for m in (0, 17, 39):
        h1, y1, _ = forward(L, x[m : m + 1], p, None, 0.0)
        assert float((y1.double() - y[m : m + 1].double()).norm() / y[m].double().norm()) < 2.0 ** -8 * 3
        a = L.block_join_fwd(x[m : m + 1], h[m : m + 1], post_gamma=p["gp"], pre_gamma=p["g1"])
        b = L.block_join_fwd(x, h, post_gamma=p["gp"], pre_gamma=p["g1"])
        assert torch.equal(a[0][0], b[0][m]) and torch.equal(a[1][0], b[1][m])


def test_two_streams_at_once(L):
    """Two steps at the same time, each with scratch of its own, give what they give alone."""
    M, C, F = 700, 512, 1368
    p = weights(C, F)
    data = [(draw(M, C, 30 + i), draw(M, C, 40 + i, 0.1), draw(M, C, 50 + i, 0.1)) for i in range(2)]
    rng = L.dropout_rng(9)

    def step(x, dh, dy):
        h, y, kept = forward(L, x, p, rng, 0.1)
        return [h, y] + list(backward(L, dh, dy, kept, p).values())

    want = [step(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = []
    for s, d in zip(streams, data):
        with torch.cuda.stream(s):
            got.append([step(*d) for _ in range(5)])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, r))
