"""The 16/32-bit operators' argument checks at the C ABI (CPU only: every call is refused, or has no
rows, before anything is enqueued), their structs' layouts and their size queries."""
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


def ck(L, **kw):
    c = L.CCkpt(FAKE, FAKE, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_scale_pitch(L):
    assert [L.act_ckpt_scale_pitch(n) for n in (0, 1, 128, 129, 2048, -1)] == [0, 4, 4, 8, 64, -1]


@pytest.mark.parametrize("args,status,needle", [
    (dict(elem=3), 1, "elem"), (dict(rows=-1), 1, "rows"), (dict(cols=0), 2, "cols"), (dict(ldx=5), 1, "ldx"),
    (dict(x=None), 1, "x is NULL"), (dict(x=FAKE + 1), 1, "2-byte"), (dict(c=dict(codes=None)), 1, "NULL"),
    (dict(c=dict(dtype=2)), 1, "dtype"), (dict(c=dict(scales=FAKE + 2)), 1, "4-byte"), (dict(rows=1 << 31), 2, "rows"),
])
def test_save_refuses(L, args, status, needle):
    a = dict(x=FAKE, elem=0, rows=4, cols=64, ldx=0)
    c = ck(L, **args.pop("c", {}))
    a.update(args)
    assert L._c_ckpt_save(a["x"], a["elem"], a["rows"], a["cols"], a["ldx"], ctypes.byref(c), None) == status
    assert needle in L.last_error()


@pytest.mark.parametrize("args,status,needle", [
    (dict(act=4), 1, "act"), (dict(gamma=FAKE), 1, "together"), (dict(gamma=FAKE, beta=FAKE, act=1), 5, "activation"),
    (dict(gamma=FAKE, beta=FAKE, pe=9), 1, "param_elem"), (dict(out=None), 1, "out"), (dict(elem=2, out=FAKE + 2), 1, "4-byte"),
    (dict(cols=-3), 2, "cols"), (dict(ldo=1), 1, "ldo"),
])
def test_restore_refuses(L, args, status, needle):
    a = dict(rows=4, cols=64, act=0, gamma=None, beta=None, pe=0, out=FAKE, elem=0, ldo=0)
    a.update(args)
    assert L._c_ckpt_restore(ctypes.byref(ck(L)), a["rows"], a["cols"], a["act"], a["gamma"], a["beta"], a["pe"], a["out"],
                             a["elem"], a["ldo"], None) == status
    assert needle in L.last_error()


def ln_fwd(L, **kw):
    a = L.CLayerNormFwd(M=4, D=64, elem=0, param_elem=2, x=FAKE, gamma=FAKE, beta=FAKE, y=FAKE, mu=FAKE, rsigma=FAKE, eps=1e-5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("args,status,needle", [
    (dict(D=16385), 2, "D"), (dict(D=0), 2, "D"), (dict(M=-2), 1, "M"), (dict(elem=7), 1, "elem"), (dict(param_elem=-1), 1, "param_elem"),
    (dict(gamma=FAKE + 2), 1, "gamma"), (dict(beta=None), 1, "beta"), (dict(residual=FAKE), 1, "x_sum"), (dict(eps=-1.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"), (dict(ldy=63), 1, "ldy"), (dict(mu=None), 1, "mu"),
])
def test_layernorm_fwd_refuses(L, args, status, needle):
    assert L._c_layernorm_fwd(ctypes.byref(ln_fwd(L, **args)), None) == status
    assert needle in L.last_error()


def test_layernorm_fwd_refuses_half_a_checkpoint(L):
    a = ln_fwd(L)
    a.ckpt = ck(L, codes=None)
    assert L._c_layernorm_fwd(ctypes.byref(a), None) == 1 and "ckpt" in L.last_error()
    assert L._c_layernorm_fwd(ctypes.byref(ln_fwd(L, M=0, x=None, y=None)), None) == 0


@pytest.mark.parametrize("args,status,needle", [
    (dict(workspace_bytes=16), 1, "workspace"), (dict(workspace=None), 1, "workspace"), (dict(workspace=FAKE + 4), 1, "workspace"),
    (dict(x=None), 1, "x is NULL"), (dict(mu=None), 1, "mu"), (dict(rsigma=None), 1, "rsigma"), (dict(dgamma=None), 1, "dgamma"),
    (dict(ld_dy=10), 1, "ld_dy"), (dict(ld_dresidual=10), 1, "ld_dresidual"), (dict(D=20000), 2, "D"),
])
def test_layernorm_bwd_refuses(L, args, status, needle):
    a = L.CLayerNormBwd(M=4, D=64, elem=0, param_elem=0, dy=FAKE, x=FAKE, mu=FAKE, rsigma=FAKE, gamma=FAKE, dx=FAKE, dgamma=FAKE,
                        dbeta=FAKE, workspace=FAKE, workspace_bytes=1 << 30)
    for k, v in args.items():
        setattr(a, k, v)
    assert L._c_layernorm_bwd(ctypes.byref(a), None) == status
    assert needle in L.last_error()
    a.ckpt = ck(L)
    if not args.keys() & {"x", "mu"}:
        return
    assert L.layernorm_bwd_workspace_size(-1, 4) == -1 and L.layernorm_bwd_workspace_size(0, 4) == 0


def test_layernorm_bwd_refuses_both_sources(L):
    a = L.CLayerNormBwd(M=4, D=64, elem=0, param_elem=0, dy=FAKE, x=FAKE, mu=FAKE, rsigma=FAKE, gamma=FAKE, dx=FAKE, dgamma=FAKE,
                        dbeta=FAKE, workspace=FAKE, workspace_bytes=1 << 30, ckpt=ck(L))
    assert L._c_layernorm_bwd(ctypes.byref(a), None) == 1 and "checkpoint" in L.last_error()


@pytest.mark.parametrize("args,status,needle", [
    (dict(elem=2), 1, "elem"), (dict(act=9), 1, "act"), (dict(K=12), 2, "multiple of 8"), (dict(N=0), 2, "N"), (dict(M=-1), 1, "M"),
    (dict(x=FAKE + 8), 1, "x is not 16-byte"), (dict(bias=FAKE + 2), 1, "bias"), (dict(ldx=66), 1, "ldx"), (dict(ldy=32), 1, "ldy"),
    (dict(w=None), 1, "w is NULL"), (dict(y=None), 1, "y is NULL"), (dict(residual=FAKE + 4), 1, "residual"),
])
def test_linear_act_fwd_refuses(L, args, status, needle):
    a = L.CLinearActFwd(M=4, K=64, N=64, x=FAKE, w=FAKE, y=FAKE)
    for k, v in args.items():
        setattr(a, k, v)
    assert L._c_linear_act_fwd(ctypes.byref(a), None) == status
    assert needle in L.last_error()


def test_linear_act_fwd_refuses_checkpoints(L):
    a = L.CLinearActFwd(M=4, K=64, N=64, x=FAKE, w=FAKE, y=FAKE, h=FAKE, ckpt=ck(L))
    assert L._c_linear_act_fwd(ctypes.byref(a), None) == 1 and "checkpoint" in L.last_error()
    a = L.CLinearActFwd(M=4, K=64, N=64, x=FAKE, w=FAKE, y=FAKE, ckpt=ck(L, codes=FAKE + 4))
    assert L._c_linear_act_fwd(ctypes.byref(a), None) == 1 and "8-byte" in L.last_error()
    a = L.CLinearActFwd(M=0, K=64, N=64, w=FAKE)
    assert L._c_linear_act_fwd(ctypes.byref(a), None) == 0


@pytest.mark.parametrize("args,status,needle", [
    (dict(elem=2), 1, "elem"), (dict(act=1, h=None), 1, "h is NULL"), (dict(x=None), 1, "x is NULL"), (dict(x_act=1), 1, "checkpoint"),
    (dict(x_act=8), 1, "x_act"), (dict(workspace=None), 1, "workspace"), (dict(workspace_bytes=8), 1, "workspace"),
    (dict(w=None), 1, "w is NULL"), (dict(ld_dy=60), 1, "ld_dy"), (dict(dw=FAKE + 2), 1, "dw"), (dict(x_gamma=FAKE), 1, "checkpoint"),
    (dict(N=4), 2, "multiple of 8"), (dict(dbias=FAKE + 2), 1, "dbias"),
])
def test_linear_act_bwd_refuses(L, args, status, needle):
    a = L.CLinearActBwd(M=4, K=64, N=64, dy=FAKE, x=FAKE, w=FAKE, h=FAKE, dx=FAKE, dw=FAKE, dbias=FAKE, workspace=FAKE,
                        workspace_bytes=1 << 40)
    for k, v in args.items():
        setattr(a, k, v)
    assert L._c_linear_act_bwd(ctypes.byref(a), None) == status
    assert needle in L.last_error()


def test_linear_act_bwd_refuses_checkpoint_mixes(L):
    def call(**kw):
        a = L.CLinearActBwd(M=4, K=64, N=64, dy=FAKE, x=None, w=FAKE, dx=FAKE, dw=FAKE, x_ckpt=ck(L), workspace=FAKE,
                            workspace_bytes=1 << 40)
        for k, v in kw.items():
            setattr(a, k, v)
        return L._c_linear_act_bwd(ctypes.byref(a), None)

    assert call(x=FAKE) == 1 and "checkpoint" in L.last_error()
    assert call(x_gamma=FAKE) == 1 and "together" in L.last_error()
    assert call(x_gamma=FAKE, x_beta=FAKE, x_act=1) == 5
    assert L.linear_act_bwd_workspace_size(-1, 8, 8, has_act=True, x_from_ckpt=False) == -1
    small, big = (L.linear_act_bwd_workspace_size(100, 64, 96, has_act=a, x_from_ckpt=a) for a in (False, True))
    assert small >= 96 * 4 and big >= small + 100 * (64 + 96) * 2


@pytest.mark.parametrize("M", [(1 << 31) - 1, (1 << 31) - 1023])
def test_linear_act_refuses_more_tokens_than_its_tiles_count(L, M):
    """Rows of a tile are 32-bit numbers up to a tile past the last token."""
    f = L.CLinearActFwd(M=M, K=64, N=64, x=FAKE, w=FAKE, y=FAKE)
    assert L._c_linear_act_fwd(ctypes.byref(f), None) == 2 and "M" in L.last_error()
    b = L.CLinearActBwd(M=M, K=64, N=64, dy=FAKE, x=FAKE, w=FAKE, dx=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=1 << 60)
    assert L._c_linear_act_bwd(ctypes.byref(b), None) == 2 and "M" in L.last_error()


def test_linear_act_bwd_refuses_both_forms_of_h(L):
    a = L.CLinearActBwd(M=4, K=64, N=64, act=1, dy=FAKE, x=FAKE, w=FAKE, h=FAKE, h_ckpt=ck(L), dx=FAKE, dw=FAKE, workspace=FAKE,
                        workspace_bytes=1 << 40)
    assert L._c_linear_act_bwd(ctypes.byref(a), None) == 1 and "h and a checkpoint" in L.last_error()


@pytest.mark.parametrize("name", ["K", "N"])
def test_linear_act_refuses_more_features_than_its_sums_count(L, name):
    """The backward's two column sums of N, rounded up to whole blocks of 32, are a 32-bit number."""
    for v in (1 << 30, (1 << 30) - 24):
        f = L.CLinearActFwd(M=4, K=64, N=64, x=FAKE, w=FAKE, y=FAKE)
        b = L.CLinearActBwd(M=4, K=64, N=64, dy=FAKE, x=FAKE, w=FAKE, dx=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=1 << 60)
        for a, call in ((f, L._c_linear_act_fwd), (b, L._c_linear_act_bwd)):
            setattr(a, name, v)
            assert call(ctypes.byref(a), None) == 2 and f"{name} = {v}" in L.last_error()
    f = L.CLinearActFwd(M=0, K=64, N=64, w=FAKE)
    setattr(f, name, (1 << 30) - 32)
    assert L._c_linear_act_fwd(ctypes.byref(f), None) == 0


STRUCTS = {"lnfp8_ckpt": "CCkpt", "lnfp8_layernorm_fwd_args": "CLayerNormFwd", "lnfp8_layernorm_bwd_args": "CLayerNormBwd",
           "lnfp8_linear_act_fwd_args": "CLinearActFwd", "lnfp8_linear_act_bwd_args": "CLinearActBwd"}


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
