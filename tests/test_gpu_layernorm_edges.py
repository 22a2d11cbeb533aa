"""layernorm_bwd (GPU) of row groups that get few rows or none, behind a call that leaves other statistics in the shared memory
that theirs are copied to. Bounds as in test_gpu_layernorm_rows.py."""
import pytest

torch = pytest.importorskip("torch")
import plain64 as P  # noqa: E402
from test_gpu_layernorm_rows import DTYPES, check_bwd, draw, params  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 3, 37, 305, 1300])
@pytest.mark.parametrize("cols", [16, 128, 512, 2048, 8192])
@pytest.mark.parametrize("ckpt", [False, True])
def test_statistics_behind_another_call(L, rows, cols, dtype, ckpt):
    gamma, beta = params(cols, dtype)
    far = draw(1300, cols, dtype, 7, 4.0, 50.0)
    x, dy, dres = draw(rows, cols, dtype, 1), draw(rows, cols, dtype, 5, 0.1), draw(rows, cols, dtype, 6, 0.1)
    before = L.layernorm_fwd(far, gamma, beta, ckpt=ckpt)[1]
    ctx = L.layernorm_fwd(x, gamma, beta, ckpt=ckpt)[1]
    L.layernorm_bwd(far, before, gamma, dresidual=far)
    g = L.layernorm_bwd(dy, ctx, gamma, dresidual=dres)
    rs = ctx.rsigma.double()
    if ckpt:
        xh = P.decode(ctx.ckpt.codes, ctx.ckpt.scales, 0)
        dxh = torch.zeros_like(xh)
    else:
        xh = (x.double() - ctx.mu.double()[:, None]) * rs[:, None]
        dxh = 2.01 * P.U * xh.abs()
    check_bwd(g, dy, xh, dxh, rs, gamma, dres)
