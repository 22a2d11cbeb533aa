"""What a transformer block runs beside its plain linear layers, as a training or serving program calls it: the gated
linear layer of a feed-forward block (forward, backward), the join of a block's output with the residual stream (norm
after the block, gate, dropout, residual scale, norm before the next block; forward, backward), and dropout alone
(forward, backward).

Each case is one call. `run` computes it either from elementary torch operations in fp32 (`own` false) or through the
framework's entry points (`own` true); `exact` gives the same outputs from the definitions in fp64.

Definitions.
  gated linear   z = x w^T + b with w [2N, K], gate rows first; y = act(z_gate) z_up; z is kept in the type.
                 Backward: dz_gate = dy z_up act'(z_gate), dz_up = dy act(z_gate), dx = dz w, dw = dz^T x, db = sum dz.
  join           n = norm(x) post_gamma + post_beta, t = gate n, h = r + scale drop(t), rounded to the type and kept,
                 y = norm(h) pre_gamma + pre_beta; every part may be left out. norm: (v - mean) / sqrt(var + eps), or
                 v / sqrt(mean(v^2) + eps).
  dropout        element (row, col) draws 16 bits u and is dropped where u < t = round(65536 p), else multiplied by
                 65536 / (65536 - t). The bits are Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as
                 1, 2, 3", 2011) with the key seed and the counter (col / 8, row, step, site): the eight 16-bit parts of
                 its four words, low half first, belong to eight neighbouring columns. (seed, step) is a device tensor."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the feed-forward block of one decoded token: the weight's bytes
        {"name": "glu_fwd_1x2048x8192_bf16_silu", "op": "glu_fwd", "m": 1, "k": 2048, "n": 8192, "dtype": "bf16", "act": "silu", "bias": False, "save": False},
        # a short ragged batch through a small model's block
        {"name": "glu_fwd_333x768x2048_f16_gelu", "op": "glu_fwd", "m": 333, "k": 768, "n": 2048, "dtype": "f16", "act": "gelu", "bias": True, "save": False},
        # a training step's forward, pre-activations kept
        {"name": "glu_fwd_8192x2048x8192_bf16_silu_kept", "op": "glu_fwd", "m": 8192, "k": 2048, "n": 8192, "dtype": "bf16", "act": "silu", "bias": False, "save": True},
        # a training step's backward at the usual two thirds of four times the width
        {"name": "glu_bwd_8192x2048x5504_bf16_silu", "op": "glu_bwd", "m": 8192, "k": 2048, "n": 5504, "dtype": "bf16", "act": "silu", "bias": False},
        # the backward of a small model over a ragged batch
        {"name": "glu_bwd_1000x768x2048_f16_gelu", "op": "glu_bwd", "m": 1000, "k": 768, "n": 2048, "dtype": "f16", "act": "gelu", "bias": True},
        # between two blocks while decoding one token: launch latency
        {"name": "join_fwd_1x2048_bf16", "op": "join_fwd", "rows": 1, "cols": 2048, "dtype": "bf16", "norm": "rms", "beta": False, "post": True, "gate": False, "pre": True, "scale": 1.0, "p": 0.0},
        # between two blocks of a training step: norms on both sides and dropout
        {"name": "join_fwd_16384x2048_bf16_drop", "op": "join_fwd", "rows": 16384, "cols": 2048, "dtype": "bf16", "norm": "rms", "beta": False, "post": True, "gate": False, "pre": True, "scale": 1.0, "p": 0.1},
        # a layer-normalised model of odd width, its output gated and scaled
        {"name": "join_fwd_4099x1001_f16_layer_gate", "op": "join_fwd", "rows": 4099, "cols": 1001, "dtype": "f16", "norm": "layer", "beta": True, "post": False, "gate": True, "pre": True, "scale": 0.5, "p": 0.0},
        # the training step's backward between two blocks
        {"name": "join_bwd_16384x2048_bf16_drop", "op": "join_bwd", "rows": 16384, "cols": 2048, "dtype": "bf16", "norm": "rms", "beta": False, "post": True, "gate": False, "pre": True, "scale": 1.0, "p": 0.1},
        # the same kept in fp32, layer-normalised with a gate, an odd number of tokens
        {"name": "join_bwd_8191x768_f32_layer_gate", "op": "join_bwd", "rows": 8191, "cols": 768, "dtype": "f32", "norm": "layer", "beta": True, "post": False, "gate": True, "pre": True, "scale": 0.5, "p": 0.0},
        # dropout of a small batch
        {"name": "drop_fwd_77x2304_f16", "op": "drop_fwd", "rows": 77, "cols": 2304, "dtype": "f16", "p": 0.1},
        # the backward of a dropout behind a wide activation
        {"name": "drop_bwd_16384x8192_bf16", "op": "drop_bwd", "rows": 16384, "cols": 8192, "dtype": "bf16", "p": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glu_fwd", "glu_bwd", "join_fwd", "join_bwd", "drop_fwd", "drop_bwd"])
    if op.startswith("glu"):
        while True:
            m, k, n = _log(rng, 1, 16384), 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
            if m * k * n <= (1 << 36 if op == "glu_bwd" else 1 << 37):
                break
        c = {"op": op, "m": m, "k": k, "n": n, "dtype": rng.choice(["bf16", "f16"]),
             "act": rng.choice(["none", "gelu", "relu", "silu"]), "bias": rng.random() < 0.5}
        if op == "glu_fwd":
            c["save"] = rng.random() < 0.5
        return c
    join = op.startswith("join")
    while True:
        rows, cols = _log(rng, 1, 65536), _log(rng, 16, 16384)
        if rng.random() < 0.5:
            cols = max(8, cols // 8 * 8)
        if rows * cols <= (1 << 25 if join else 1 << 27):
            break
    c = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f16", "f32"])}
    if join:
        c["norm"] = rng.choice(["rms", "layer"])
        for part in ("beta", "post", "gate", "pre"):
            c[part] = rng.random() < 0.6
        c["scale"] = rng.choice([1.0, 0.5, 0.22])
        c["p"] = rng.choice([0.0, 0.1, 0.3])
    else:
        c["p"] = rng.choice([0.05, 0.1, 0.3, 0.5])
    return c


def work(case):
    s = SIZE[case["dtype"]]
    if case["op"].startswith("glu"):
        m, k, n = case["m"], case["k"], case["n"]
        if case["op"] == "glu_fwd":
            b = 2 * s * n if case["bias"] else 0
            return {"bytes": s * (m * k + 2 * n * k + m * n * (3 if case["save"] else 1)) + b, "flops": 4 * m * n * k}
        return {"bytes": s * (3 * m * n + 2 * m * k + 4 * n * k) + (8 * n if case["bias"] else 0), "flops": 8 * m * n * k}
    r, d = case["rows"], case["cols"]
    if case["op"].startswith("drop"):
        return {"bytes": 2 * s * r * d, "flops": 2 * r * d}
    params = sum((1 + case["beta"]) * case[part] for part in ("post", "pre")) + case["gate"]
    stats = 4 * r * (2 if case["norm"] == "layer" else 1) * (case["post"] + case["pre"])
    if case["op"] == "join_fwd":
        return {"bytes": s * r * d * (4 if case["pre"] else 3) + s * d * params + stats, "flops": 12 * r * d}
    tensors = 3 + (2 if case["pre"] else 0) + (1 if case["post"] or case["gate"] else 0)
    return {"bytes": s * r * d * tensors + (s + 4) * d * params + stats, "flops": 24 * r * d}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dt)

    def hidden(*shape):  # hidden states: a few entries are much larger than the rest
        v = torch.randn(*shape, generator=g, device="cuda")
        return torch.where(torch.rand(*shape, generator=g, device="cuda") < 1e-3, v * 50, v).to(dt)

    s = {"case": case}
    if case["op"].startswith("glu"):
        m, k, n = case["m"], case["k"], case["n"]
        s["w"], s["x"] = normal(2 * n, k, std=0.02), normal(m, k)
        if case["op"] == "glu_fwd":
            if case["bias"]:
                s["b"] = normal(2 * n, std=0.02)
        else:
            s["dy"], s["z"] = normal(m, n, std=0.01), normal(m, 2 * n)
        return s
    r, d = case["rows"], case["cols"]
    s["rng"] = torch.randint(0, 1 << 31, (2,), generator=g, device="cuda")
    s["rng"][0] += torch.randint(0, 1 << 31, (1,), generator=g, device="cuda")[0] << 32
    if case["op"].startswith("drop"):
        s["x"] = hidden(r, d) if case["op"] == "drop_fwd" else normal(r, d, std=0.01)
        return s
    for part in ("post", "pre"):
        if case[part]:
            s[part + "_gamma"] = normal(d, std=0.1, mean=1.0)
            if case["beta"]:
                s[part + "_beta"] = normal(d, std=0.1)
    if case["gate"]:
        s["gate"] = normal(d, std=0.2, mean=0.5)
    s["x"] = hidden(r, d)
    if case["op"] == "join_fwd":
        s["r"] = hidden(r, d)
        return s
    s["dh"] = normal(r, d, std=0.01)
    if case["pre"]:
        s["h"], s["dy"] = hidden(r, d), normal(r, d, std=0.01)
    for part, name in (("post", "x"), ("pre", "h")):
        if case[part]:
            v = s[name].double()
            mu = v.mean(1, keepdim=True) if case["norm"] == "layer" else 0.0
            s[part + "_rs"] = torch.rsqrt((v - mu).square().mean(1) + EPS).float()
            if case["norm"] == "layer":
                s[part + "_mu"] = mu.float().reshape(-1)
    return s


SITE = 5  # of the one dropout in a case


# ------------------------------------------------------------------ the plain forms (fp32)
LOW = 0xFFFFFFFF


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _bits(rng, rows, cols):
    """The 16-bit draws [rows, cols]. 64-bit integers hold the 32-bit words; a product's high word survives the wrap."""
    groups = (cols + 7) // 8
    c0 = torch.arange(groups, device=rng.device).expand(rows, groups)
    c1 = torch.arange(rows, device=rng.device)[:, None].expand(rows, groups)
    c2, c3 = rng[1] & LOW, torch.full_like(rng[1], SITE)
    k0, k1 = rng[0] & LOW, (rng[0] >> 32) & LOW
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & LOW) ^ c1 ^ k0, b & LOW, ((a >> 32) & LOW) ^ c3 ^ k1, a & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    w = torch.stack((c0, c1, c2, c3), 2)
    return torch.stack((w & 0xFFFF, w >> 16), 3).view(rows, groups * 8)[:, :cols]


def _drop(t, rng, p):
    cut = _threshold(p)
    if cut == 0:
        return t
    return torch.where(_bits(rng, *t.shape) >= cut, t * (65536 / (65536 - cut)), torch.zeros_like(t))


def _act(z, act):
    if act == "gelu":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _dact(z, act):
    if act == "gelu":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "none":
        return torch.ones_like(z)
    s = 1 / (1 + torch.exp(-z))
    return s + z * s * (1 - s)


def _stats(v, norm):
    mu = v.mean(1, keepdim=True) if norm == "layer" else torch.zeros_like(v[:, :1])
    return mu, 1 / torch.sqrt((v - mu).square().mean(1, keepdim=True) + EPS)


def _affine(xh, s, part):
    n = xh * s[part + "_gamma"].float()
    return n + s[part + "_beta"].float() if part + "_beta" in s else n


def _hat(s, part, name):
    v = s[name].float()
    if part + "_mu" in s:
        v = v - s[part + "_mu"][:, None]
    return v * s[part + "_rs"][:, None]


def _norm_back(g, xh, rs, norm):
    g = g - xh * (g * xh).mean(1, keepdim=True) - (g.mean(1, keepdim=True) if norm == "layer" else 0.0)
    return g * rs[:, None]


def _plain(s):
    c = s["case"]
    op, dt = c["op"], TYPES[c["dtype"]]
    if op == "glu_fwd":
        z = s["x"].float() @ s["w"].float().t()
        if c["bias"]:
            z = z + s["b"].float()
        out = {"y": (_act(z[:, : c["n"]], c["act"]) * z[:, c["n"] :]).to(dt)}
        if c["save"]:
            out["z"] = z.to(dt)
        return out
    if op == "glu_bwd":
        dy, zg, zu = s["dy"].float(), s["z"][:, : c["n"]].float(), s["z"][:, c["n"] :].float()
        dz = torch.cat((dy * zu * _dact(zg, c["act"]), dy * _act(zg, c["act"])), 1)
        out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt)}
        if c["bias"]:
            out["db"] = dz.sum(0)
        return out
    if op.startswith("drop"):
        return _drop(s["x"].float(), s["rng"], c["p"]).to(dt)
    if op == "join_fwd":
        out = {}
        t = s["x"].float()
        if c["post"]:
            mu, rs = _stats(t, c["norm"])
            out["post_rs"] = rs.reshape(-1)
            t = _affine((t - mu) * rs, s, "post")
        if c["gate"]:
            t = t * s["gate"].float()
        h = out["h"] = (s["r"].float() + c["scale"] * _drop(t, s["rng"], c["p"])).to(dt)
        if c["pre"]:
            v = h.float()
            mu, rs = _stats(v, c["norm"])
            out["pre_rs"], out["y"] = rs.reshape(-1), _affine((v - mu) * rs, s, "pre").to(dt)
        return out
    out = {}
    dh = s["dh"].float()
    if c["pre"]:
        dy, hh = s["dy"].float(), _hat(s, "pre", "h")
        dh = dh + _norm_back(dy * s["pre_gamma"].float(), hh, s["pre_rs"], c["norm"])
        out["dpre_gamma"] = (dy * hh).sum(0)
        if c["beta"]:
            out["dpre_beta"] = dy.sum(0)
    out["dr"] = dh.to(dt)
    dn = dt_ = c["scale"] * _drop(dh, s["rng"], c["p"])
    if c["gate"]:
        dn = dt_ * s["gate"].float()
    if c["post"]:
        xh = _hat(s, "post", "x")
        out["dpost_gamma"] = (dn * xh).sum(0)
        if c["beta"]:
            out["dpost_beta"] = dn.sum(0)
        if c["gate"]:
            out["dgate"] = (dt_ * _affine(xh, s, "post")).sum(0)
        out["dx"] = _norm_back(dn * s["post_gamma"].float(), xh, s["post_rs"], c["norm"]).to(dt)
    else:
        if c["gate"]:
            out["dgate"] = (dt_ * s["x"].float()).sum(0)
        out["dx"] = dn.to(dt)
    return out


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from fp8_delayed_scaling_row_gb300 import lnfp8 as L

    c = s["case"]
    op = c["op"]
    if op == "glu_fwd":
        y, ctx = L.linear_glu_fwd(s["x"], s["w"], s.get("b"), act=c["act"], save="h" if c["save"] else "none")
        return {"y": y, "z": ctx.h} if c["save"] else {"y": y}
    if op == "glu_bwd":
        g = L.linear_glu_bwd(s["dy"], s["x"], s["w"], L.LinearGluCtx(act=c["act"], h=s["z"]), dbias=c["bias"])
        out = {"dx": g.dx, "dw": g.dw}
        if c["bias"]:
            out["db"] = g.dbias
        return out
    if op == "drop_fwd":
        return L.dropout_fwd(s["x"], c["p"], s["rng"], site=SITE)[0]
    if op == "drop_bwd":
        return L.dropout_bwd(s["x"], L.DropoutCtx(p=c["p"], rng=s["rng"], site=SITE))
    params = {k: s.get(k) for k in ("post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta")}
    if op == "join_fwd":
        h, y, ctx = L.block_join_fwd(s["x"], s["r"], norm=c["norm"], scale=c["scale"], eps=EPS, p=c["p"], rng=s["rng"], site=SITE, **params)
        out = {"h": h}
        if c["post"]:
            out["post_rs"] = ctx.post_rsigma
        if c["pre"]:
            out["pre_rs"], out["y"] = ctx.pre_rsigma, y
        return out
    ctx = L.BlockJoinCtx(x=s["x"], h=s.get("h"), norm=c["norm"], scale=c["scale"], p=c["p"], rng=s["rng"], site=SITE,
                         post_mu=s.get("post_mu"), post_rsigma=s.get("post_rs"), pre_mu=s.get("pre_mu"), pre_rsigma=s.get("pre_rs"))
    g = L.block_join_bwd(s["dh"], s.get("dy"), ctx, **params)
    out = {"dr": g.dresidual, "dx": g.dx}
    out.update({"d" + k: getattr(g, "d" + k) for k, v in params.items() if v is not None})
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in fp64
def _exact_keep(rng, rows, cols, p):
    """The factor of each element: 0, or 65536 / (65536 - t). Philox by 16-bit halves: no product passes 2^33."""
    key, step = (int(v) for v in rng.tolist())

    def times(word, m):
        lo, hi = word & 0xFFFF, word >> 16
        a, b, d = lo * (m & 0xFFFF), lo * (m >> 16), hi * (m & 0xFFFF)
        mid = (a >> 16) + (b & 0xFFFF) + (d & 0xFFFF)
        return hi * (m >> 16) + (b >> 16) + (d >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) | (a & 0xFFFF)

    groups = -(-cols // 8)
    ctr = [torch.arange(groups, device="cuda").repeat(rows), torch.arange(rows, device="cuda").repeat_interleave(groups)]
    ctr += [torch.full_like(ctr[0], step % 2 ** 32), torch.full_like(ctr[0], SITE)]
    for i in range(10):
        k = [(key % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32, (key // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32]
        (h0, l0), (h1, l1) = times(ctr[0], 0xD2511F53), times(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ k[0], l1, h0 ^ ctr[3] ^ k[1], l0]
    draws = torch.empty(rows * groups, 8, dtype=torch.int64, device="cuda")
    for j in range(8):
        draws[:, j] = (ctr[j // 2] >> (16 * (j % 2))) & 0xFFFF
    t = round(p * 65536)
    kept = draws.reshape(rows, groups * 8)[:, :cols] >= t
    return kept.to(torch.float64) * (65536.0 / (65536 - t))


def _exact_act(z, act):
    """The activation and its slope."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).to(z.dtype)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = lambda name: s[name].to(torch.float64)  # noqa: E731
    if op == "glu_fwd":
        z = torch.mm(f("x"), f("w").t())
        if case["bias"]:
            z += f("b")
        gate, up = z.chunk(2, dim=1)
        out = {"y": _exact_act(gate, case["act"])[0] * up}
        if case["save"]:
            out["z"] = z
        return out
    if op == "glu_bwd":
        gate, up = f("z").chunk(2, dim=1)
        a, slope = _exact_act(gate, case["act"])
        dg, du = f("dy") * up * slope, f("dy") * a
        wg, wu = f("w").chunk(2, dim=0)
        out = {"dx": dg @ wg + du @ wu, "dw": torch.cat((dg.t() @ f("x"), du.t() @ f("x")))}
        if case["bias"]:
            out["db"] = torch.cat((dg.sum(0), du.sum(0)))
        return out
    keep = _exact_keep(s["rng"], case["rows"], case["cols"], case["p"])
    if op.startswith("drop"):
        return f("x") * keep
    d, layer = case["cols"], case["norm"] == "layer"

    def normed(v, part):
        dev = v - v.sum(1, keepdim=True) / d if layer else v
        rs = ((dev * dev).sum(1) / d + EPS) ** -0.5
        return rs, dev * rs[:, None] * f(part + "_gamma") + (f(part + "_beta") if case["beta"] else 0.0)

    def given(part, name):
        return (f(name) - f(part + "_mu")[:, None] if layer else f(name)) * f(part + "_rs")[:, None]

    def back(g, xh, rs):
        total = xh * (g * xh).sum(1, keepdim=True)
        if layer:
            total = total + g.sum(1, keepdim=True)
        return rs[:, None] * (g - total / d)

    if op == "join_fwd":
        out, t = {}, f("x")
        if case["post"]:
            out["post_rs"], t = normed(t, "post")
        if case["gate"]:
            t = t * f("gate")
        out["h"] = f("r") + t * keep * case["scale"]
        if case["pre"]:  # normalised as it is kept
            out["pre_rs"], out["y"] = normed(out["h"].to(TYPES[case["dtype"]]).to(torch.float64), "pre")
        return out
    out, dh = {}, f("dh")
    if case["pre"]:
        hh = given("pre", "h")
        dh = dh + back(f("dy") * f("pre_gamma"), hh, f("pre_rs"))
        out["dpre_gamma"] = (f("dy") * hh).sum(0)
        if case["beta"]:
            out["dpre_beta"] = f("dy").sum(0)
    out["dr"] = dh
    d_t = dh * keep * case["scale"]
    gate = f("gate") if case["gate"] else 1.0
    if case["post"]:
        xh = given("post", "x")
        n = xh * f("post_gamma") + (f("post_beta") if case["beta"] else 0.0)
        out["dpost_gamma"] = (d_t * gate * xh).sum(0)
        if case["beta"]:
            out["dpost_beta"] = (d_t * gate).sum(0)
        out["dx"] = back(d_t * gate * f("post_gamma"), xh, f("post_rs"))
    else:
        n = f("x")
        out["dx"] = d_t * gate
    if case["gate"]:
        out["dgate"] = (d_t * n).sum(0)
    return out
