"""8-bit activation checkpoints (GPU): act_ckpt_save bit for bit against the definition in 64 bits,
act_ckpt_restore exact, or within its roundings through an activation or gamma and beta."""
import pytest

torch = pytest.importorskip("torch")
import plain64 as P  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def hidden(rows, cols, dtype, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(rows, cols, generator=g, device="cuda") * std
    return torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 1e-2, v * 50, v).to(dtype)


def check_saved(ck, x, fmt):
    cols = x.shape[1]
    want = P.scale_bytes(x, fmt)
    assert torch.equal(ck.scales[:, : want.shape[1]], want)
    scale = torch.exp2(want.double() - 127).repeat_interleave(32, 1)[:, :cols]
    ok = (want != 255).repeat_interleave(32, 1)[:, :cols]
    v = (x.double() / scale).float()  # a power of two: exact, and within the format's range
    codes = torch.where(ok, v, torch.zeros_like(v)).to(P.F8[fmt]).float()
    got = ck.codes.view(P.F8[fmt]).float()
    assert torch.equal(got[ok], codes[ok])
    assert torch.isnan(got[~ok]).all()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (3, 31), (5, 33), (7, 1001), (64, 768), (33, 136), (2, 8200), (300, 40)])
def test_save_matches_the_definition(L, rows, cols, dtype, fmt):
    x = hidden(rows, cols, dtype, seed=rows + cols)
    check_saved(L.act_ckpt_save(x, dtype=fmt), x, fmt)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
def test_save_at_the_borders(L, dtype, fmt):
    """Blocks whose largest value sits on, just below and just above fmax 2^k; zeros; the type's extremes;
    subnormals; ties of the code grid; blocks with Inf or NaN, which come back as NaN throughout."""
    fi = torch.finfo(dtype)
    x = hidden(24, 64, dtype, seed=5)
    top = torch.tensor(1.75, dtype=dtype, device="cuda")
    for i, k in enumerate((0, 3, 9)):
        at = top * 2.0 ** k
        x[3 * i, :32] = x[3 * i, :32].clamp(-1, 1)
        x[3 * i, 5] = at
        x[3 * i + 1, 7] = at * 4 * (1 + fi.eps)
        x[3 * i + 2, 9] = -at * 4 * (1 - fi.eps)
    x[9] = 0
    x[10] = -0.0
    x[11, 3], x[11, 40] = fi.max, -fi.max
    x[12] = fi.smallest_normal * fi.eps * torch.arange(64, device="cuda")  # subnormals
    x[13] = (torch.arange(64, device="cuda") / 16 + 1).to(dtype)           # ties between codes
    x[14, 2], x[15, 40], x[16, 3], x[16, 4] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[17] = fi.tiny
    check_saved(L.act_ckpt_save(x, dtype=fmt), x, fmt)
    back = L.act_ckpt_restore(L.act_ckpt_save(x, dtype=fmt), out_dtype=dtype)
    assert torch.isfinite(back[:14]).all() and torch.isfinite(back[17:]).all()
    assert torch.isnan(back[14, :32]).all() and torch.isfinite(back[14, 32:]).all()
    assert torch.isnan(back[15, 32:]).all() and torch.isfinite(back[15, :32]).all()
    assert torch.equal(back[9], x[9])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 33), (9, 1001), (40, 768), (3, 8200), (65, 136)])
@pytest.mark.parametrize("act", ["none", "gelu", "relu", "silu"])
def test_restore(L, rows, cols, out_dtype, fmt, act):
    ck = L.act_ckpt_save(hidden(rows, cols, torch.bfloat16, seed=cols), dtype=fmt)
    z = P.decode(ck.codes, ck.scales, fmt)
    out = L.act_ckpt_restore(ck, out_dtype=out_dtype, act=act)
    want = P.act(z, act)
    # none, relu: the code times a power of two is exact in fp32. gelu, silu: z s(u) with ex2.approx and
    # rcp.approx (2 ulp each) and u rounded 4 times, which moves s by |u| 4 U (1 - s) relative; where s itself
    # underflows (u < -87) fp32 gives 0 for a value below 87 2^-126
    u = 1.6 * (z.abs() + 0.045 * z.abs() ** 3) if act == "gelu" else z.abs()
    soft = (16 + 4 * u.clamp(max=90)) * P.U * want.abs() + 1e-35 if act in ("gelu", "silu") else 0
    P.assert_within(out, want, soft + P.half(out_dtype) * want.abs() + P.tiny(out_dtype), act)


@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("pdtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(3, 33), (20, 768)])
def test_restore_with_gamma_and_beta(L, rows, cols, out_dtype, pdtype):
    ck = L.act_ckpt_save(hidden(rows, cols, torch.bfloat16, seed=3))
    gamma, beta = hidden(1, cols, pdtype, seed=8)[0], hidden(1, cols, pdtype, seed=9)[0]
    out = L.act_ckpt_restore(ck, out_dtype=out_dtype, gamma=gamma, beta=beta)
    want = P.decode(ck.codes, ck.scales, 0) * gamma.double() + beta.double()
    P.assert_within(out, want, (P.half(out_dtype) + P.U) * 1.001 * want.abs() + P.tiny(out_dtype), "affine")


def test_restore_saturates_and_keeps_nan(L):
    x = torch.full((4, 32), 1e30, dtype=torch.float32, device="cuda")
    x[1] = -1e30
    x[2, 5] = float("nan")
    x[3] = 3.4e38  # rounds up past the largest fp32
    ck = L.act_ckpt_save(x)
    out = L.act_ckpt_restore(ck, out_dtype=torch.float16)
    assert (out[0] == 65504).all() and (out[1] == -65504).all() and torch.isnan(out[2]).all() and (out[3] == 65504).all()
    for dt in (torch.float32, torch.bfloat16):
        assert (L.act_ckpt_restore(ck, out_dtype=dt)[3] == torch.finfo(dt).max).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_alignment_and_neighbours(L, dtype):
    """Rows inside a wider tensor, from an odd column on; what lies around the outputs stays."""
    wide = hidden(37, 200, dtype, seed=2)
    for lo, cols in ((0, 136), (1, 130), (3, 64), (8, 128)):
        x = wide[:, lo : lo + cols]
        a, b = L.act_ckpt_save(x), L.act_ckpt_save(x.contiguous())
        nb = (cols + 31) // 32
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales[:, :nb], b.scales[:, :nb])
        buf = torch.full((39, 200), 7.0, dtype=dtype, device="cuda")
        out = buf[1:38, lo : lo + cols]
        L.act_ckpt_restore(a, out=out)
        assert torch.equal(out, L.act_ckpt_restore(a, out_dtype=dtype))
        buf[1:38, lo : lo + cols] = 7.0
        assert (buf == 7.0).all()
    codes = torch.full((6, 136), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((6, 8), 9, dtype=torch.uint8, device="cuda")
    L.act_ckpt_save(hidden(4, 136, dtype), ckpt=L.ActCkpt(codes[1:5], scales[1:5]))
    assert (codes[[0, 5]] == 9).all() and (scales[[0, 5]] == 9).all()


def test_no_rows(L):
    ck = L.act_ckpt_save(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert L.act_ckpt_restore(ck).shape == (0, 64)


def test_offsets_past_32_bits(L):
    rows, cols = 66000, 32776
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = hidden(3, cols, torch.bfloat16, seed=11)
    x[-3:] = tail
    ck = L.act_ckpt_save(x)
    check_saved(L.ActCkpt(ck.codes[-3:], ck.scales[-3:]), tail, 0)
    assert not ck.codes[:-3].any()
    out = L.act_ckpt_restore(ck, out=x)
    assert torch.equal(out[-3:], L.act_ckpt_restore(L.ActCkpt(ck.codes[-3:], ck.scales[-3:]))) and not out[:-3].any()


def test_stream_and_graph(L):
    x = hidden(100, 768, torch.bfloat16, seed=4)
    want = L.act_ckpt_restore(L.act_ckpt_save(x), act="gelu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = L.act_ckpt_restore(L.act_ckpt_save(x, stream=s), act="gelu", stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = L.act_ckpt_restore(L.act_ckpt_save(x), act="gelu")
    x.copy_(hidden(100, 768, torch.bfloat16, seed=5))
    g.replay()
    assert torch.equal(got, L.act_ckpt_restore(L.act_ckpt_save(x), act="gelu"))


def test_binding_refuses(L):
    x = hidden(4, 64, torch.bfloat16)
    ck = L.act_ckpt_save(x)
    with pytest.raises(TypeError):
        L.act_ckpt_save(x.double())
    with pytest.raises(TypeError):
        L.act_ckpt_save(x.cpu())
    with pytest.raises(ValueError):
        L.act_ckpt_save(x[0])
    with pytest.raises(ValueError):
        L.act_ckpt_save(x.t())
    with pytest.raises(ValueError):
        L.act_ckpt_save(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        L.act_ckpt_save(x, ckpt=L.act_ckpt(4, 32))
    with pytest.raises(ValueError):
        L.act_ckpt_restore(ck, act="tanh")
    with pytest.raises(L.LnFp8Error):
        L.act_ckpt_restore(ck, gamma=x[0])
    with pytest.raises(L.LnFp8Error):
        L.act_ckpt_restore(ck, gamma=x[0], beta=x[0], act="gelu")
