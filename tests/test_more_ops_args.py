"""Argument checks of the gated linear layer, the join of a block's output and dropout at the C ABI (CPU only: every call
is refused, or has no rows, before anything is enqueued), their structs' layouts and their size queries."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    from fp8_delayed_scaling_row_gb300.build import LIB, build_library
    if not os.path.exists(LIB):
        build_library()
    from fp8_delayed_scaling_row_gb300 import lnfp8
    return lnfp8


def glu_fwd(L, **kw):
    return L.CLinearGluFwd(**{**dict(M=4, K=64, N=64, x=FAKE, w=FAKE, y=FAKE), **kw})


@pytest.mark.parametrize("args,status,needle", [
    (dict(elem=2), 1, "elem"), (dict(act=4), 1, "act"), (dict(K=12), 2, "multiple of 8"), (dict(N=0), 2, "N"), (dict(N=(1 << 29) - 8), 2, "N"),
    (dict(M=-1), 1, "M"), (dict(M=(1 << 31) - 1023), 2, "M"), (dict(x=FAKE + 8), 1, "x is not 16-byte"), (dict(bias=FAKE + 2), 1, "bias"),
    (dict(ldx=66), 1, "ldx"), (dict(ldy=32), 1, "ldy"), (dict(w=None), 1, "w is NULL"), (dict(y=None), 1, "y is NULL"), (dict(h=FAKE + 4), 1, "h"),
])
def test_linear_glu_fwd_refuses(L, args, status, needle):
    assert L._c_linear_glu_fwd(ctypes.byref(glu_fwd(L, **args)), None) == status
    assert needle in L.last_error()


def test_linear_glu_without_tokens(L):
    assert L._c_linear_glu_fwd(ctypes.byref(glu_fwd(L, M=0, x=None, y=None)), None) == 0
    assert L.linear_glu_bwd_workspace_size(0, 64, 64) == 0 and L.linear_glu_bwd_workspace_size(-1, 64, 64) == -1
    assert L.linear_glu_bwd_workspace_size(100, 64, 96) >= 100 * 192 * 2 + 192 * 4


@pytest.mark.parametrize("args,status,needle", [
    (dict(elem=2), 1, "elem"), (dict(act=-1), 1, "act"), (dict(h=None), 1, "h is NULL"), (dict(x=None), 1, "x is NULL"),
    (dict(w=None), 1, "w is NULL"), (dict(dy=None), 1, "dy is NULL"), (dict(workspace=None), 1, "workspace"), (dict(workspace_bytes=8), 1, "workspace"),
    (dict(workspace=FAKE + 8), 1, "workspace"), (dict(ld_dy=60), 1, "ld_dy"), (dict(ld_dx=68), 1, "ld_dx"), (dict(dw=FAKE + 2), 1, "dw"),
    (dict(dbias=FAKE + 2), 1, "dbias"), (dict(N=4), 2, "multiple of 8"), (dict(N=1 << 29), 2, "N"),
])
def test_linear_glu_bwd_refuses(L, args, status, needle):
    a = L.CLinearGluBwd(**{**dict(M=4, K=64, N=64, dy=FAKE, x=FAKE, w=FAKE, h=FAKE, dx=FAKE, dw=FAKE, dbias=FAKE, workspace=FAKE,
                                  workspace_bytes=1 << 40), **args})
    assert L._c_linear_glu_bwd(ctypes.byref(a), None) == status
    assert needle in L.last_error()


@pytest.mark.parametrize("args,status,needle", [
    (dict(elem=3), 1, "elem"), (dict(rows=-1), 1, "rows"), (dict(rows=1 << 31), 2, "rows"), (dict(cols=0), 2, "cols"), (dict(cols=(1 << 30) + 1), 2, "cols"),
    (dict(ldx=5), 1, "ldx"), (dict(ldy=63), 1, "ldy"), (dict(x=None), 1, "x is NULL"), (dict(y=FAKE + 1), 1, "2-byte"), (dict(p=1.5), 1, "p = 1.5"),
    (dict(p=-0.1), 1, "p = "), (dict(p=float("nan")), 1, "p = "), (dict(rng=None), 1, "rng"), (dict(rng=FAKE + 4), 1, "8-byte"),
    (dict(rng_saved=FAKE + 4), 1, "rng_saved"),
])
def test_dropout_refuses(L, args, status, needle):
    a = {**dict(x=FAKE, elem=0, rows=4, cols=64, ldx=0, y=FAKE, ldy=0, p=0.1, rng=FAKE, rng_saved=None), **args}
    d = L.CDropout(a["p"], a["rng"], a["rng_saved"], 0)
    assert L._c_dropout(a["x"], a["elem"], a["rows"], a["cols"], a["ldx"], ctypes.byref(d), a["y"], a["ldy"], None) == status
    assert needle in L.last_error()


def test_dropout_of_nothing(L):
    d = L.CDropout(0.5, FAKE, None, 0)
    assert L._c_dropout(None, 0, 0, 64, 0, ctypes.byref(d), None, 0, None) == 0
    assert L._c_dropout(FAKE, 0, 4, 64, 0, None, FAKE, 0, None) == 1 and "drop" in L.last_error()


def join_fwd(L, **kw):
    drop = L.CDropout(kw.pop("p", 0.0), kw.pop("rng", None), None, 0)
    return L.CBlockJoinFwd(**{**dict(M=4, D=64, param_elem=2, norm=1, eps=1e-5, scale=1.0, x=FAKE, residual=FAKE, post_gamma=FAKE, pre_gamma=FAKE,
                                     h=FAKE, y=FAKE, post_mu=FAKE, post_rsigma=FAKE, pre_mu=FAKE, pre_rsigma=FAKE, drop=drop), **kw})


@pytest.mark.parametrize("args,status,needle", [
    (dict(D=16385), 2, "D"), (dict(D=0), 2, "D"), (dict(M=-2), 1, "M"), (dict(elem=7), 1, "elem"), (dict(param_elem=-1), 1, "param_elem"),
    (dict(norm=2), 1, "norm"), (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(x=None), 1, "x is NULL"), (dict(h=None), 1, "h is NULL"),
    (dict(y=None), 1, "y is NULL"), (dict(post_gamma=FAKE + 2), 1, "post_gamma"), (dict(post_gamma=None, post_beta=FAKE), 1, "post_beta"),
    (dict(pre_gamma=None, pre_beta=FAKE), 1, "pre_beta"), (dict(gate=FAKE + 1), 1, "gate"), (dict(post_mu=None), 1, "post_mu"), (dict(pre_mu=None), 1, "pre_mu"),
    (dict(post_rsigma=None), 1, "post_rsigma"), (dict(pre_rsigma=None), 1, "pre_rsigma"), (dict(ldh=63), 1, "ldh"), (dict(ld_residual=2), 1, "ld_residual"),
    (dict(p=0.1), 1, "rng"), (dict(p=2.0, rng=FAKE), 1, "p = 2"), (dict(residual=FAKE + 1), 1, "residual"),
])
def test_block_join_fwd_refuses(L, args, status, needle):
    assert L._c_block_join_fwd(ctypes.byref(join_fwd(L, **args)), None) == status
    assert needle in L.last_error()


@pytest.mark.parametrize("args,status,needle", [
    (dict(workspace_bytes=16), 1, "workspace"), (dict(workspace=None), 1, "workspace"), (dict(dh=None, pre_gamma=None, dpre_gamma=None, dy=None), 1, "neither"),
    (dict(dy=None), 1, "dy is NULL"), (dict(pre_gamma=None), 1, "without pre_gamma"), (dict(pre_gamma=None, dpre_gamma=None), 1, "dy without pre_gamma"),
    (dict(x=None), 1, "x is NULL"), (dict(h=None), 1, "h is NULL"), (dict(post_rsigma=None), 1, "post_rsigma"), (dict(pre_mu=None), 1, "pre_mu"),
    (dict(dpost_gamma=None), 1, "dpost_gamma"), (dict(dgate=FAKE), 1, "dgate without"), (dict(gate=FAKE), 1, "dgate is NULL"), (dict(dpre_gamma=None), 1, "dpre_gamma"),
    (dict(post_gamma=None), 1, "without post_gamma"), (dict(post_gamma=None, dpost_gamma=None, post_beta=FAKE), 1, "post_beta"), (dict(norm=-1), 1, "norm"),
    (dict(ld_dh=60), 1, "ld_dh"), (dict(ld_dresidual=60), 1, "ld_dresidual"), (dict(dx=None), 1, "dx is NULL"), (dict(dpre_beta=FAKE + 2), 1, "dpre_beta"),
    (dict(D=20000), 2, "D"),
])
def test_block_join_bwd_refuses(L, args, status, needle):
    a = L.CBlockJoinBwd(**{**dict(M=4, D=64, param_elem=0, norm=1, scale=1.0, dh=FAKE, dy=FAKE, x=FAKE, h=FAKE, post_gamma=FAKE, pre_gamma=FAKE, post_mu=FAKE,
                                  post_rsigma=FAKE, pre_mu=FAKE, pre_rsigma=FAKE, dx=FAKE, dresidual=FAKE, dpost_gamma=FAKE, dpre_gamma=FAKE, workspace=FAKE,
                                  workspace_bytes=1 << 30), **args})
    assert L._c_block_join_bwd(ctypes.byref(a), None) == status
    assert needle in L.last_error()


def test_block_join_sizes(L):
    assert L._c_block_join_fwd(ctypes.byref(join_fwd(L, M=0, x=None, h=None, y=None, residual=None)), None) == 0
    assert L.block_join_bwd_workspace_size(-1, 4) == -1 and L.block_join_bwd_workspace_size(0, 4) == 0
    assert L.block_join_bwd_workspace_size(1, 100) >= 1600


STRUCTS = {"lnfp8_linear_glu_fwd_args": "CLinearGluFwd", "lnfp8_linear_glu_bwd_args": "CLinearGluBwd", "lnfp8_dropout": "CDropout",
           "lnfp8_block_join_fwd_args": "CBlockJoinFwd", "lnfp8_block_join_bwd_args": "CBlockJoinBwd"}


def test_struct_layouts_match_the_header(L, tmp_path):
    """A C program built on the header prints every field's offset; the ctypes mirrors agree."""
    lines, want = [], []
    for cname, pname in STRUCTS.items():
        cls = getattr(L, pname)
        lines.append(f'printf("%zu\\n", sizeof({cname}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({cname}, {f}));')
            want.append(getattr(cls, f).offset)
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"lnfp8.h\"\nint main(void) {\n" + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([shutil.which("gcc") or "cc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == want


def test_binding_refuses_on_the_host(L):
    """What the binding says before it looks at a device."""
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="expected one of"):
        L.linear_glu_fwd(torch.zeros(4, 8), torch.zeros(16, 8))
    with pytest.raises(ValueError, match="rows"):
        L.linear_glu_fwd(x, torch.zeros(15, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="save"):
        L.linear_glu_fwd(x, torch.zeros(16, 8, dtype=torch.bfloat16), save="ckpt")
    with pytest.raises(ValueError, match="norm"):
        L.block_join_fwd(x, x, norm="batch")
    with pytest.raises(ValueError, match="neither"):
        L.block_join_bwd(None, None, L.BlockJoinCtx())
    with pytest.raises(TypeError, match="not a CUDA tensor"):
        L.dropout_fwd(x, 0.5, None)
