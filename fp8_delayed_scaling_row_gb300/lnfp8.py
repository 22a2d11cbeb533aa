"""Python binding of liblnfp8 (the C ABI declared in include/lnfp8.h).

Argument marshalling only: PyTorch provides device memory and the current CUDA
stream; every step of the computation runs in the library's CUDA kernels. If
the shared library has not been built, importing this module raises.

Names follow the C ABI: lnfp8_meta_init, amax_history_update, fp8_quantize,
ln_fwd_cast, ln_bwd, fp8_gemm, ln_linear_fwd / ln_linear_bwd,
ln_mlp_fwd / ln_mlp_bwd; and, for what a model keeps in 16 or 32 bits,
layernorm_fwd / layernorm_bwd, act_ckpt_save / act_ckpt_restore and
linear_act_fwd / linear_act_bwd.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass, field

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblnfp8.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"liblnfp8.so is not built ({LIB_PATH}); run fp8_delayed_scaling_row_gb300.build.build_library()")
_lib = C.CDLL(LIB_PATH)

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, ERR_CUDA, ERR_TIMEOUT, ERR_UNSUPPORTED = range(6)
E4M3, E5M2 = 0, 1
FORMAT_E4M3, FORMAT_HYBRID, FORMAT_E5M2 = 0, 1, 2
_FORMATS = {"e4m3": FORMAT_E4M3, "hybrid": FORMAT_HYBRID, "e5m2": FORMAT_E5M2}

EXPORTED = [
    "lnfp8_last_error", "lnfp8_sync_status", "lnfp8_version", "lnfp8_selftest_timeout", "lnfp8_launch_count",
    "lnfp8_profile_enable", "lnfp8_profile_sample", "lnfp8_profile_collect", "lnfp8_profile_get", "lnfp8_meta_init", "amax_history_update", "amax_history_update_many",
    "fp8_quantize", "fp8_weight_quantize", "ln_fwd_cast", "ln_bwd", "fp8_gemm", "ln_linear_fwd", "ln_linear_bwd",
    "ln_linear_bwd_noalloc", "ln_mlp_fwd", "ln_mlp_bwd", "lnfp8_gemm_workspace_size",
    "lnfp8_ln_linear_bwd_workspace_size", "lnfp8_ln_mlp_bwd_workspace_size", "lnfp8_ln_mlp_fwd_workspace_size",
    "lnfp8_ctx_bytes", "lnfp8_ctx_offsets", "lnfp8_act_ckpt_scale_pitch", "act_ckpt_save", "act_ckpt_restore",
    "layernorm_fwd", "layernorm_bwd", "lnfp8_layernorm_bwd_workspace_size", "linear_act_fwd", "linear_act_bwd",
    "lnfp8_linear_act_bwd_workspace_size",
]
OP_LN_LINEAR, OP_LINEAR, OP_LN_MLP = 0, 1, 2


class LnFp8Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"lnfp8 status {status}: {msg}")
        self.status = status


# ------------------------------------------------------------------ C structs
class CRecipe(C.Structure):
    _fields_ = [("format", C.c_int), ("history_len", C.c_int), ("algo", C.c_int), ("margin", C.c_int)]


class CMeta(C.Structure):
    _fields_ = [("scale", C.c_void_p), ("scale_inv", C.c_void_p), ("amax_history", C.c_void_p),
                ("amax_cur", C.c_void_p), ("n", C.c_int), ("history_len", C.c_int)]


_P = C.c_void_p
_I64 = C.c_int64


class CLnLinearFwd(C.Structure):
    _fields_ = [("M", _I64), ("K", _I64), ("N", _I64), ("x", _P), ("gamma", _P), ("beta", _P), ("eps", C.c_float),
                ("w", _P), ("bias", _P), ("y", _P), ("xq", _P), ("wq", _P), ("mu", _P), ("rsigma", _P),
                ("sinv_saved", _P), ("meta", CMeta), ("recipe", CRecipe), ("defer_update", C.c_int),
                ("ln_out_debug", _P), ("w_scale_inv", _P), ("residual", _P), ("x_sum", _P), ("path", C.c_int)]


PATH_AUTO, PATH_FUSED, PATH_SEPARATE = 0, 1, 2


class CLnLinearBwd(C.Structure):
    _fields_ = [("M", _I64), ("K", _I64), ("N", _I64), ("dy", _P), ("x", _P), ("gamma", _P), ("xq", _P),
                ("wq", _P), ("mu", _P), ("rsigma", _P), ("sinv_saved", _P), ("dx", _P), ("dw", _P), ("dbias", _P),
                ("dgamma", _P), ("dbeta", _P), ("dyq", _P), ("dln", _P), ("meta", CMeta), ("recipe", CRecipe),
                ("defer_update", C.c_int), ("gemm_ws", _P), ("gemm_ws_bytes", _I64)]


class CLnMlpFwd(C.Structure):
    _fields_ = [("M", _I64), ("D", _I64), ("F", _I64), ("x", _P), ("gamma", _P), ("beta", _P), ("eps", C.c_float),
                ("w1", _P), ("b1", _P), ("w2", _P), ("b2", _P), ("y", _P), ("lnq", _P), ("mu", _P), ("rsigma", _P),
                ("w1q", _P), ("w2q", _P), ("h", _P), ("aq", _P), ("sinv_saved", _P), ("meta", CMeta),
                ("recipe", CRecipe), ("defer_update", C.c_int), ("ln_out_debug", _P), ("act_debug", _P),
                ("gemm_ws", _P), ("gemm_ws_bytes", _I64), ("w1_scale_inv", _P), ("w2_scale_inv", _P),
                ("residual", _P), ("x_sum", _P)]


class CLnMlpBwd(C.Structure):
    _fields_ = [("M", _I64), ("D", _I64), ("F", _I64), ("dy", _P), ("x", _P), ("gamma", _P), ("lnq", _P),
                ("mu", _P), ("rsigma", _P), ("w1q", _P), ("w2q", _P), ("h", _P), ("aq", _P), ("sinv_saved", _P),
                ("dx", _P), ("dgamma", _P), ("dbeta", _P), ("dw1", _P), ("db1", _P), ("dw2", _P), ("db2", _P),
                ("dyq", _P), ("dhq", _P), ("dln", _P), ("meta", CMeta), ("recipe", CRecipe),
                ("defer_update", C.c_int), ("dh_debug", _P), ("gemm_ws", _P), ("gemm_ws_bytes", _I64)]


class CCkpt(C.Structure):
    _fields_ = [("codes", _P), ("scales", _P), ("dtype", C.c_int)]


class CLayerNormFwd(C.Structure):
    _fields_ = [("M", _I64), ("D", _I64), ("elem", C.c_int), ("param_elem", C.c_int), ("x", _P), ("residual", _P),
                ("gamma", _P), ("beta", _P), ("y", _P), ("x_sum", _P), ("mu", _P), ("rsigma", _P), ("ckpt", CCkpt),
                ("ldx", _I64), ("ld_residual", _I64), ("ldy", _I64), ("eps", C.c_float)]


class CLayerNormBwd(C.Structure):
    _fields_ = [("M", _I64), ("D", _I64), ("elem", C.c_int), ("param_elem", C.c_int), ("dy", _P), ("x", _P), ("mu", _P),
                ("rsigma", _P), ("ckpt", CCkpt), ("gamma", _P), ("dresidual", _P), ("dx", _P), ("dgamma", _P),
                ("dbeta", _P), ("workspace", _P), ("workspace_bytes", _I64), ("ld_dy", _I64), ("ldx", _I64),
                ("ld_dresidual", _I64), ("ld_dx", _I64)]


class CLinearActFwd(C.Structure):
    _fields_ = [("M", _I64), ("K", _I64), ("N", _I64), ("elem", C.c_int), ("act", C.c_int), ("x", _P), ("w", _P),
                ("bias", _P), ("residual", _P), ("y", _P), ("h", _P), ("ckpt", CCkpt), ("ldx", _I64),
                ("ld_residual", _I64), ("ldy", _I64)]


class CLinearActBwd(C.Structure):
    _fields_ = [("M", _I64), ("K", _I64), ("N", _I64), ("elem", C.c_int), ("act", C.c_int), ("dy", _P), ("x", _P),
                ("x_ckpt", CCkpt), ("x_act", C.c_int), ("x_gamma", _P), ("x_beta", _P), ("w", _P), ("h", _P),
                ("h_ckpt", CCkpt), ("dx", _P), ("dw", _P), ("dbias", _P), ("workspace", _P), ("workspace_bytes", _I64),
                ("ld_dy", _I64), ("ldx", _I64), ("ld_dx", _I64)]


def _sig(name, args, res=C.c_int):
    f = getattr(_lib, name)
    f.argtypes = args
    f.restype = res
    return f


_lib.lnfp8_last_error.restype = C.c_char_p
_lib.lnfp8_last_error.argtypes = []
_c_sync = _sig("lnfp8_sync_status", [_P])
_c_version = _sig("lnfp8_version", [])
_c_selftest = _sig("lnfp8_selftest_timeout", [_I64, _P])
_c_launch_count = _sig("lnfp8_launch_count", [], C.c_longlong)
_c_prof_enable = _sig("lnfp8_profile_enable", [C.c_int])
_c_prof_sample = _sig("lnfp8_profile_sample", [])
_c_prof_collect = _sig("lnfp8_profile_collect", [])
_c_prof_get = _sig("lnfp8_profile_get", [C.c_int, C.POINTER(C.c_char_p), C.POINTER(C.c_double),
                                         C.POINTER(C.c_longlong)])
_c_meta_init = _sig("lnfp8_meta_init", [C.POINTER(CMeta), _P])
_c_update = _sig("amax_history_update", [C.POINTER(CMeta), C.POINTER(CRecipe), C.POINTER(C.c_int), _P, _P])
_c_update_many = _sig("amax_history_update_many", [C.POINTER(CMeta), C.c_int, C.POINTER(CRecipe), C.POINTER(C.c_int),
                                                   C.POINTER(_P), _P])
_c_quant = _sig("fp8_quantize", [_P, C.c_int, _I64, _I64, C.c_int, _P, _P, _P, _P, _P, _P])
_c_wquant = _sig("fp8_weight_quantize", [_P, _I64, _I64, C.POINTER(CMeta), C.POINTER(CRecipe), C.c_int, _P, _P])
_c_ln_fwd = _sig("ln_fwd_cast", [_P, _P, _P, C.c_float, _I64, _I64, C.c_int, _P, _P, _P, _P, _P, _P, _P])
_c_ln_bwd = _sig("ln_bwd", [_P, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P])
_c_gemm = _sig("fp8_gemm", [_P, C.c_int, C.c_int, _P, C.c_int, C.c_int, _I64, _I64, _I64, _P, _P, _P, _P, _P, _I64,
                            _P])
_c_gemm_ws = _sig("lnfp8_gemm_workspace_size", [_I64, _I64, _I64], C.c_int64)
_c_lin_bwd_ws = _sig("lnfp8_ln_linear_bwd_workspace_size", [_I64, _I64, _I64], C.c_int64)
_c_mlp_bwd_ws = _sig("lnfp8_ln_mlp_bwd_workspace_size", [_I64, _I64, _I64], C.c_int64)
_c_mlp_fwd_ws = _sig("lnfp8_ln_mlp_fwd_workspace_size", [_I64, _I64, _I64], C.c_int64)
_c_ctx_bytes = _sig("lnfp8_ctx_bytes", [C.c_int, _I64, _I64, _I64], C.c_int64)
_c_ctx_offsets = _sig("lnfp8_ctx_offsets", [C.c_int, _I64, _I64, _I64, C.POINTER(_I64), C.c_int], C.c_int)
_c_lin_fwd = _sig("ln_linear_fwd", [C.POINTER(CLnLinearFwd), _P])
_c_lin_bwd = _sig("ln_linear_bwd", [C.POINTER(CLnLinearBwd), _P])
_c_lin_bwd_noalloc = _sig("ln_linear_bwd_noalloc", [C.POINTER(CLnLinearBwd), _P])
_c_mlp_fwd = _sig("ln_mlp_fwd", [C.POINTER(CLnMlpFwd), _P])
_c_mlp_bwd = _sig("ln_mlp_bwd", [C.POINTER(CLnMlpBwd), _P])
_c_ckpt_save = _sig("act_ckpt_save", [_P, C.c_int, _I64, _I64, _I64, C.POINTER(CCkpt), _P])
_c_ckpt_restore = _sig("act_ckpt_restore", [C.POINTER(CCkpt), _I64, _I64, C.c_int, _P, _P, C.c_int, _P, C.c_int, _I64, _P])
_c_ckpt_pitch = _sig("lnfp8_act_ckpt_scale_pitch", [_I64], C.c_int64)
_c_layernorm_fwd = _sig("layernorm_fwd", [C.POINTER(CLayerNormFwd), _P])
_c_layernorm_bwd = _sig("layernorm_bwd", [C.POINTER(CLayerNormBwd), _P])
_c_linear_act_fwd = _sig("linear_act_fwd", [C.POINTER(CLinearActFwd), _P])
_c_linear_act_bwd = _sig("linear_act_bwd", [C.POINTER(CLinearActBwd), _P])
_c_linear_act_bwd_ws = _sig("lnfp8_linear_act_bwd_workspace_size", [_I64, _I64, _I64, C.c_int, C.c_int], C.c_int64)
_c_layernorm_bwd_ws = _sig("lnfp8_layernorm_bwd_workspace_size", [_I64, _I64], C.c_int64)


def _check(st: int) -> None:
    if st != OK:
        raise LnFp8Error(st, _lib.lnfp8_last_error().decode())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def version() -> int:
    return _c_version()


def last_error() -> str:
    return _lib.lnfp8_last_error().decode()


def lnfp8_selftest_timeout(limit_ns: int, stream=None) -> None:
    """Enqueue the bounded-wait diagnostic; the next sync_status() raises ERR_TIMEOUT."""
    _check(_c_selftest(int(limit_ns), _stream(stream)))


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(_c_launch_count())


def profile_enable(on: bool = True) -> None:
    """Per-kernel CUDA-event timing on the launching stream (discards old records)."""
    _check(_c_prof_enable(int(on)))


def profile_sample() -> None:
    """After a replay of a graph captured with profiling on: add its kernel times to the totals."""
    _check(_c_prof_sample())


def profile_collect() -> dict:
    """{kernel kind: (total_ms, launches)} for everything recorded since profile_enable."""
    n = _c_prof_collect()
    out = {}
    for i in range(n):
        k, ms, cnt = C.c_char_p(), C.c_double(), C.c_longlong()
        _check(_c_prof_get(i, C.byref(k), C.byref(ms), C.byref(cnt)))
        out[k.value.decode()] = (ms.value, cnt.value)
    return out


def sync_status(stream=None) -> None:
    """Synchronise and raise if a bounded device wait has given up since the last check."""
    _check(_c_sync(_stream(stream)))


# ------------------------------------------------------------------ state
@dataclass
class Recipe:
    """DelayedScaling(fp8_format, amax_history_len, amax_compute_algo) of the TE tutorial."""
    fp8_format: str = "hybrid"
    amax_history_len: int = 16
    amax_compute_algo: str = "max"
    margin: int = 0

    def c(self) -> CRecipe:
        if self.amax_compute_algo != "max":
            raise ValueError("only amax_compute_algo='max' is supported")
        return CRecipe(_FORMATS[self.fp8_format], self.amax_history_len, 0, self.margin)

    @property
    def fwd_dtype(self) -> int:
        return E5M2 if self.fp8_format == "e5m2" else E4M3

    @property
    def bwd_dtype(self) -> int:
        return E4M3 if self.fp8_format == "e4m3" else E5M2


class ScalingMeta:
    """Device-resident delayed-scaling state of n FP8 tensors (one fp8_meta
    direction): scale [n], scale_inv [n], amax_history [L, n], amax_cur [n]."""

    def __init__(self, n: int, history_len: int, device="cuda", stream=None):
        self.n, self.history_len = n, history_len
        self.scale = torch.empty(n, dtype=torch.float32, device=device)
        self.scale_inv = torch.empty(n, dtype=torch.float32, device=device)
        self.amax_history = torch.empty(history_len, n, dtype=torch.float32, device=device)
        self.amax_cur = torch.empty(n, dtype=torch.float32, device=device)
        lnfp8_meta_init(self, stream)

    def c(self) -> CMeta:
        return CMeta(self.scale.data_ptr(), self.scale_inv.data_ptr(), self.amax_history.data_ptr(),
                     self.amax_cur.data_ptr(), self.n, self.history_len)

    def state_dict(self) -> dict:
        return {k: getattr(self, k).clone() for k in ("scale", "scale_inv", "amax_history", "amax_cur")}

    def load_state_dict(self, sd: dict) -> None:
        for k in ("scale", "scale_inv", "amax_history", "amax_cur"):
            getattr(self, k).copy_(sd[k])


def lnfp8_meta_init(meta: ScalingMeta, stream=None) -> None:
    cm = meta.c()
    _check(_c_meta_init(C.byref(cm), _stream(stream)))


def amax_history_update(meta: ScalingMeta, recipe: Recipe, dtypes, scale_inv_before=None, stream=None) -> None:
    arr = (C.c_int * meta.n)(*[int(d) for d in dtypes])
    cm, cr = meta.c(), recipe.c()
    _check(_c_update(C.byref(cm), C.byref(cr), arr, _ptr(scale_inv_before), _stream(stream)))


# ------------------------------------------------------------------ kernels

def amax_history_update_many(metas, recipe: Recipe, dtypes_per_meta, scale_inv_before=None, stream=None) -> None:
    """One launch of the state update for several ScalingMeta sets (e.g. all layers after a step)."""
    metas = list(metas)
    arr = (CMeta * len(metas))(*[m.c() for m in metas])
    flat = [int(d) for ds in dtypes_per_meta for d in ds]
    if len(flat) != sum(m.n for m in metas):
        raise ValueError("one dtype per slot of every meta")
    dts = (C.c_int * max(len(flat), 1))(*flat)
    sinv = None
    if scale_inv_before is not None:
        sinv = (_P * len(metas))(*[_ptr(t) for t in scale_inv_before])
    rc = recipe.c()
    _check(_c_update_many(arr, len(metas), C.byref(rc), dts, sinv, _stream(stream)))

def fp8_quantize(x, dtype, scale, amax_cur, *, out=None, out_t=None, colsum=None, stream=None):
    """codes = fp8(x * scale) with amax; x is a 2-D bf16 or fp32 CUDA tensor."""
    rows, cols = x.shape
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("fp8_quantize takes bf16 or fp32 input")
    _check(_c_quant(_ptr(x), int(x.dtype == torch.float32), rows, cols, dtype, _ptr(scale), _ptr(amax_cur),
                    _ptr(out), _ptr(out_t), _ptr(colsum), _stream(stream)))
    return out, out_t, colsum


@dataclass
class FP8Weight:
    """A weight kept as FP8 codes (fp8_model_init): codes [rows, cols] uint8 in the
    recipe's forward format, and the weight's own state (n = 1), whose scale_inv
    [1] is the codes' dequantisation factor."""
    codes: torch.Tensor
    meta: "ScalingMeta"
    dtype: int

    @property
    def scale_inv(self) -> torch.Tensor:
        return self.meta.scale_inv

    @property
    def shape(self):
        return self.codes.shape


def quantize_weight(w, recipe: Recipe, *, meta: ScalingMeta | None = None, codes=None, stream=None) -> FP8Weight:
    """Converts a bf16 weight [rows, cols] to FP8 storage once, on the device: its
    amax, the delayed-scaling state update of its own state, then the cast."""
    rows, cols = w.shape
    if w.dtype != torch.bfloat16:
        raise TypeError("quantize_weight takes a bf16 weight")
    meta = meta if meta is not None else ScalingMeta(1, 1, device=w.device, stream=stream)
    codes = codes if codes is not None else _e((rows, cols), torch.uint8, w.device)
    dt = recipe.fwd_dtype
    cm, cr = meta.c(), recipe.c()
    _check(_c_wquant(_ptr(w), rows, cols, C.byref(cm), C.byref(cr), dt, _ptr(codes), _stream(stream)))
    return FP8Weight(codes=codes, meta=meta, dtype=dt)


def ln_fwd_cast(x, gamma, beta, dtype, scale, amax_cur, *, eps=1e-5, out=None, mu=None, rsigma=None, y_debug=None,
                stream=None):
    M, D = x.shape
    dev = x.device
    out = out if out is not None else torch.empty(M, D, dtype=torch.uint8, device=dev)
    mu = mu if mu is not None else torch.empty(M, dtype=torch.float32, device=dev)
    rsigma = rsigma if rsigma is not None else torch.empty(M, dtype=torch.float32, device=dev)
    _check(_c_ln_fwd(_ptr(x), _ptr(gamma), _ptr(beta), eps, M, D, dtype, _ptr(scale), _ptr(amax_cur), _ptr(out),
                     _ptr(mu), _ptr(rsigma), _ptr(y_debug), _stream(stream)))
    return out, mu, rsigma


def ln_bwd(dy, x, gamma, mu, rsigma, *, dx=None, dgamma=None, dbeta=None, stream=None):
    M, D = x.shape
    dev = x.device
    dx = dx if dx is not None else torch.empty(M, D, dtype=torch.bfloat16, device=dev)
    dgamma = dgamma if dgamma is not None else torch.empty(D, dtype=torch.float32, device=dev)
    dbeta = dbeta if dbeta is not None else torch.empty(D, dtype=torch.float32, device=dev)
    _check(_c_ln_bwd(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(mu), _ptr(rsigma), M, D, _ptr(dx), _ptr(dgamma),
                     _ptr(dbeta), _stream(stream)))
    return dx, dgamma, dbeta


def gemm_workspace_size(M, N, K) -> int:
    """Bytes of workspace with which fp8_gemm splits K for this shape (0: it would not)."""
    return int(_c_gemm_ws(M, N, K))


def ln_linear_bwd_workspace_size(M, K, N) -> int:
    return int(_c_lin_bwd_ws(M, K, N))


def ln_mlp_bwd_workspace_size(M, D, F) -> int:
    return int(_c_mlp_bwd_ws(M, D, F))


def ln_mlp_fwd_workspace_size(M, D, F) -> int:
    return int(_c_mlp_fwd_ws(M, D, F))


def _ws(nbytes, device):
    return torch.zeros(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None


def fp8_gemm(a, a_layout, a_dtype, b, b_layout, b_dtype, M, N, K, sinv_a, sinv_b, *, bias=None, out=None,
             workspace=None, stream=None):
    """out[M, N] bf16 = (A . B^T) * sinv_a * sinv_b + bias; layouts as in the C ABI. With a
    uint8 workspace tensor of gemm_workspace_size(M, N, K) bytes the GEMM may split K."""
    out = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=b.device)
    _check(_c_gemm(_ptr(a), a_layout, a_dtype, _ptr(b), b_layout, b_dtype, M, N, K, _ptr(sinv_a), _ptr(sinv_b),
                   _ptr(bias), _ptr(out), _ptr(workspace), workspace.numel() if workspace is not None else 0,
                   _stream(stream)))
    return out


# ------------------------------------------------------------------ modules
@dataclass
class LinearCtx:
    xq: torch.Tensor
    wq: torch.Tensor
    mu: torch.Tensor | None
    rsigma: torch.Tensor | None
    sinv_saved: torch.Tensor
    ln_out_debug: torch.Tensor | None = None
    x_sum: torch.Tensor | None = None  # h = bf16(x + residual) of a forward with a residual (the backward's x)


def _e(shape, dtype, dev):
    return torch.empty(shape, dtype=dtype, device=dev)


def ctx_bytes(op: int, M: int, D: int, F: int) -> int:
    return int(_c_ctx_bytes(op, M, D, F))


def ctx_offsets(op: int, M: int, D: int, F: int) -> list:
    """Start of each saved-context buffer, then the total (the library's layout)."""
    off = (_I64 * 9)()
    n = int(_c_ctx_offsets(op, M, D, F, off, 9))
    if n < 0:
        raise LnFp8Error(ERR_INVALID_ARG, f"lnfp8_ctx_offsets({op}, {M}, {D}, {F})")
    return [int(off[i]) for i in range(n + 1)]


def _carve(op, M, D, F, shapes, device):
    """The saved context as views of one allocation laid out by lnfp8_ctx_offsets;
    shapes: (shape, dtype) per buffer in the library's order."""
    off = ctx_offsets(op, M, D, F)
    buf = torch.empty(off[-1], dtype=torch.uint8, device=device)
    views = []
    for (shape, dtype), start in zip(shapes, off):
        nbytes = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        views.append(buf[start:start + nbytes].view(dtype).view(shape))
    return buf, views


def linear_ctx(M, K, N, *, ln=True, device="cuda", debug=False, weight_codes=True) -> LinearCtx:
    """Saved tensors of one LayerNormLinear / Linear forward, views of one allocation in
    the library's saved-context layout (weight_codes=False leaves wq to an FP8Weight)."""
    u8, f32 = torch.uint8, torch.float32
    if ln:
        _, (xq, wq, mu, rs, sinv) = _carve(OP_LN_LINEAR, M, K, N, [((M, K), u8), ((N, K), u8), ((M,), f32),
                                                                   ((M,), f32), ((2,), f32)], device)
    else:
        _, (xq, wq, sinv) = _carve(OP_LINEAR, M, K, N, [((M, K), u8), ((N, K), u8), ((2,), f32)], device)
        mu = rs = None
    return LinearCtx(xq=xq, wq=wq if weight_codes else None, mu=mu, rsigma=rs, sinv_saved=sinv,
                     ln_out_debug=_e((M, K), torch.float32, device) if debug else None)


def ln_linear_fwd(x, gamma, beta, w, bias, meta: ScalingMeta, recipe: Recipe, *, eps=1e-5, y=None,
                  ctx: LinearCtx | None = None, defer_update=False, debug=False, residual=None, path=PATH_AUTO,
                  stream=None):
    """LayerNormLinear (gamma given) or Linear (gamma None) forward; returns (y, ctx).
    w is a bf16 weight (cast every call) or an FP8Weight (its codes are used as they are).
    residual: optional bf16 [M, K]; the input becomes h = bf16(x + residual), returned as
    ctx.x_sum (pass it as the backward's x). path: PATH_AUTO, PATH_FUSED (one launch for
    the LayerNorm, casts and GEMM; K <= 768) or PATH_SEPARATE."""
    M, K = x.shape
    N = w.shape[0]
    dev = x.device
    w8 = isinstance(w, FP8Weight)
    ctx = ctx if ctx is not None else linear_ctx(M, K, N, ln=gamma is not None, device=dev, debug=debug,
                                                 weight_codes=not w8)
    if w8:
        ctx.wq = w.codes
    if residual is not None and ctx.x_sum is None:
        ctx.x_sum = _e((M, K), torch.bfloat16, dev)
    y = y if y is not None else _e((M, N), torch.bfloat16, dev)
    a = CLnLinearFwd(M=M, K=K, N=N, x=_ptr(x), gamma=_ptr(gamma), beta=_ptr(beta), eps=eps,
                     w=None if w8 else _ptr(w), bias=_ptr(bias), y=_ptr(y), xq=_ptr(ctx.xq), wq=_ptr(ctx.wq),
                     mu=_ptr(ctx.mu), rsigma=_ptr(ctx.rsigma), sinv_saved=_ptr(ctx.sinv_saved), meta=meta.c(),
                     recipe=recipe.c(), defer_update=int(defer_update), ln_out_debug=_ptr(ctx.ln_out_debug),
                     w_scale_inv=_ptr(w.scale_inv) if w8 else None, residual=_ptr(residual),
                     x_sum=_ptr(ctx.x_sum) if residual is not None else None, path=int(path))
    _check(_c_lin_fwd(C.byref(a), _stream(stream)))
    return y, ctx


@dataclass
class LinearGrads:
    dx: torch.Tensor
    dw: torch.Tensor
    dbias: torch.Tensor | None
    dgamma: torch.Tensor | None
    dbeta: torch.Tensor | None
    dyq: torch.Tensor
    dln: torch.Tensor | None
    gemm_ws: torch.Tensor | None = None  # split-K workspace of the GEMMs (None: unsplit)


def linear_grads(M, K, N, *, ln=True, bias=True, split_k=True, device="cuda") -> LinearGrads:
    return LinearGrads(dx=_e((M, K), torch.bfloat16, device), dw=_e((N, K), torch.bfloat16, device),
                       dbias=_e((N,), torch.float32, device) if bias else None,
                       dgamma=_e((K,), torch.float32, device) if ln else None,
                       dbeta=_e((K,), torch.float32, device) if ln else None,
                       dyq=_e((M, N), torch.uint8, device), dln=_e((M, K), torch.bfloat16, device) if ln else None,
                       gemm_ws=_ws(ln_linear_bwd_workspace_size(M, K, N), device) if split_k else None)


def ln_linear_bwd(dy, x, gamma, ctx: LinearCtx, meta: ScalingMeta, recipe: Recipe, *, grads: LinearGrads | None = None,
                  bias=True, defer_update=False, stream=None) -> LinearGrads:
    M, N = dy.shape
    K = x.shape[1]
    g = grads if grads is not None else linear_grads(M, K, N, ln=gamma is not None, bias=bias, device=dy.device)
    a = CLnLinearBwd(M=M, K=K, N=N, dy=_ptr(dy), x=_ptr(x), gamma=_ptr(gamma), xq=_ptr(ctx.xq), wq=_ptr(ctx.wq),
                     mu=_ptr(ctx.mu), rsigma=_ptr(ctx.rsigma), sinv_saved=_ptr(ctx.sinv_saved), dx=_ptr(g.dx),
                     dw=_ptr(g.dw), dbias=_ptr(g.dbias), dgamma=_ptr(g.dgamma), dbeta=_ptr(g.dbeta),
                     dyq=_ptr(g.dyq), dln=_ptr(g.dln), meta=meta.c(), recipe=recipe.c(),
                     defer_update=int(defer_update), gemm_ws=_ptr(g.gemm_ws),
                     gemm_ws_bytes=g.gemm_ws.numel() if g.gemm_ws is not None else 0)
    _check(_c_lin_bwd(C.byref(a), _stream(stream)))
    return g


def ln_linear_bwd_noalloc(dy, x, gamma, ctx: LinearCtx, meta: ScalingMeta, recipe: Recipe, *, dx, dw, dbias=None,
                          dgamma=None, dbeta=None, defer_update=False, stream=None) -> None:
    """LayerNormLinear backward for callers that cannot allocate device memory:
    the caller passes inputs and outputs only; the library's built-in scratch
    array holds the dY codes and the LayerNorm-output gradient (see the C
    header for its size limit and sharing rules)."""
    M, N = dy.shape
    K = x.shape[1]
    a = CLnLinearBwd(M=M, K=K, N=N, dy=_ptr(dy), x=_ptr(x), gamma=_ptr(gamma), xq=_ptr(ctx.xq), wq=_ptr(ctx.wq),
                     mu=_ptr(ctx.mu), rsigma=_ptr(ctx.rsigma), sinv_saved=_ptr(ctx.sinv_saved), dx=_ptr(dx),
                     dw=_ptr(dw), dbias=_ptr(dbias), dgamma=_ptr(dgamma), dbeta=_ptr(dbeta), dyq=None, dln=None,
                     meta=meta.c(), recipe=recipe.c(), defer_update=int(defer_update))
    _check(_c_lin_bwd_noalloc(C.byref(a), _stream(stream)))


@dataclass
class MlpCtx:
    lnq: torch.Tensor
    mu: torch.Tensor
    rsigma: torch.Tensor
    w1q: torch.Tensor
    w2q: torch.Tensor
    h: torch.Tensor
    aq: torch.Tensor
    sinv_saved: torch.Tensor
    ln_out_debug: torch.Tensor | None = None
    act_debug: torch.Tensor | None = None
    gemm_ws: torch.Tensor | None = None  # FC1 tiles' readiness counters (FC1 and FC2 in one launch)
    x_sum: torch.Tensor | None = None  # h = bf16(x + residual) of a forward with a residual (the backward's x)


def mlp_ctx(M, D, F, *, device="cuda", debug=False, fused=False, weight_codes=True) -> MlpCtx:
    """Saved tensors of one LayerNormMLP forward. fused=True also allocates the row-block
    readiness counters with which the forward runs FC1 and FC2 as one launch (same
    results; the two launches measured faster at 8192 x 768 -> 3072 -> 768 and at
    d 2048 from 8192 to 65536 tokens, equal at 2048).
    weight_codes=False leaves w1q/w2q to FP8-stored weights."""
    u8, f32 = torch.uint8, torch.float32
    _, (lnq, w1q, w2q, h, aq, mu, rs, sinv) = _carve(
        OP_LN_MLP, M, D, F, [((M, D), u8), ((F, D), u8), ((D, F), u8), ((M, F), torch.bfloat16), ((M, F), u8),
                             ((M,), f32), ((M,), f32), ((4,), f32)], device)
    return MlpCtx(lnq=lnq, mu=mu, rsigma=rs, w1q=w1q if weight_codes else None, w2q=w2q if weight_codes else None,
                  h=h, aq=aq, sinv_saved=sinv,
                  ln_out_debug=_e((M, D), torch.float32, device) if debug else None,
                  act_debug=_e((M, F), torch.float32, device) if debug else None,
                  gemm_ws=_ws(ln_mlp_fwd_workspace_size(M, D, F), device) if fused else None)


def ln_mlp_fwd(x, gamma, beta, w1, b1, w2, b2, meta: ScalingMeta, recipe: Recipe, *, eps=1e-5, y=None,
               ctx: MlpCtx | None = None, defer_update=False, debug=False, residual=None, stream=None):
    """LayerNormMLP forward; returns (y, ctx). w1 and w2 are both bf16 weights (cast
    every call) or both FP8Weight (their codes are used as they are). residual: optional
    bf16 [M, D]; the input becomes h = bf16(x + residual), returned as ctx.x_sum."""
    M, D = x.shape
    F = w1.shape[0]
    dev = x.device
    w8 = isinstance(w1, FP8Weight)
    if w8 != isinstance(w2, FP8Weight):
        raise TypeError("w1 and w2 must both be FP8Weight or both bf16")
    ctx = ctx if ctx is not None else mlp_ctx(M, D, F, device=dev, debug=debug, weight_codes=not w8)
    if w8:
        ctx.w1q, ctx.w2q = w1.codes, w2.codes
    if residual is not None and ctx.x_sum is None:
        ctx.x_sum = _e((M, D), torch.bfloat16, dev)
    y = y if y is not None else _e((M, D), torch.bfloat16, dev)
    a = CLnMlpFwd(M=M, D=D, F=F, x=_ptr(x), gamma=_ptr(gamma), beta=_ptr(beta), eps=eps,
                  w1=None if w8 else _ptr(w1), b1=_ptr(b1), w2=None if w8 else _ptr(w2), b2=_ptr(b2), y=_ptr(y),
                  lnq=_ptr(ctx.lnq), mu=_ptr(ctx.mu), rsigma=_ptr(ctx.rsigma),
                  w1q=_ptr(ctx.w1q), w2q=_ptr(ctx.w2q), h=_ptr(ctx.h), aq=_ptr(ctx.aq),
                  sinv_saved=_ptr(ctx.sinv_saved), meta=meta.c(), recipe=recipe.c(), defer_update=int(defer_update),
                  ln_out_debug=_ptr(ctx.ln_out_debug), act_debug=_ptr(ctx.act_debug), gemm_ws=_ptr(ctx.gemm_ws),
                  gemm_ws_bytes=ctx.gemm_ws.numel() if ctx.gemm_ws is not None else 0,
                  w1_scale_inv=_ptr(w1.scale_inv) if w8 else None, w2_scale_inv=_ptr(w2.scale_inv) if w8 else None,
                  residual=_ptr(residual), x_sum=_ptr(ctx.x_sum) if residual is not None else None)
    _check(_c_mlp_fwd(C.byref(a), _stream(stream)))
    return y, ctx


@dataclass
class MlpGrads:
    dx: torch.Tensor
    dgamma: torch.Tensor
    dbeta: torch.Tensor
    dw1: torch.Tensor
    db1: torch.Tensor | None
    dw2: torch.Tensor
    db2: torch.Tensor | None
    dyq: torch.Tensor
    dhq: torch.Tensor
    dln: torch.Tensor
    dh_debug: torch.Tensor | None = None
    gemm_ws: torch.Tensor | None = None  # split-K workspace of the GEMMs (None: unsplit)


def mlp_grads(M, D, F, *, bias=True, split_k=True, device="cuda", debug=False) -> MlpGrads:
    return MlpGrads(dx=_e((M, D), torch.bfloat16, device), dgamma=_e((D,), torch.float32, device),
                    dbeta=_e((D,), torch.float32, device), dw1=_e((F, D), torch.bfloat16, device),
                    db1=_e((F,), torch.float32, device) if bias else None, dw2=_e((D, F), torch.bfloat16, device),
                    db2=_e((D,), torch.float32, device) if bias else None, dyq=_e((M, D), torch.uint8, device),
                    dhq=_e((M, F), torch.uint8, device), dln=_e((M, D), torch.bfloat16, device),
                    dh_debug=_e((M, F), torch.float32, device) if debug else None,
                    gemm_ws=_ws(ln_mlp_bwd_workspace_size(M, D, F), device) if split_k else None)


def ln_mlp_bwd(dy, x, gamma, ctx: MlpCtx, meta: ScalingMeta, recipe: Recipe, *, grads: MlpGrads | None = None,
               bias=True, defer_update=False, debug=False, stream=None) -> MlpGrads:
    M, D = dy.shape
    F = ctx.h.shape[1]
    g = grads if grads is not None else mlp_grads(M, D, F, bias=bias, device=dy.device, debug=debug)
    a = CLnMlpBwd(M=M, D=D, F=F, dy=_ptr(dy), x=_ptr(x), gamma=_ptr(gamma), lnq=_ptr(ctx.lnq), mu=_ptr(ctx.mu),
                  rsigma=_ptr(ctx.rsigma), w1q=_ptr(ctx.w1q), w2q=_ptr(ctx.w2q), h=_ptr(ctx.h), aq=_ptr(ctx.aq),
                  sinv_saved=_ptr(ctx.sinv_saved), dx=_ptr(g.dx), dgamma=_ptr(g.dgamma), dbeta=_ptr(g.dbeta),
                  dw1=_ptr(g.dw1), db1=_ptr(g.db1), dw2=_ptr(g.dw2), db2=_ptr(g.db2), dyq=_ptr(g.dyq),
                  dhq=_ptr(g.dhq), dln=_ptr(g.dln), meta=meta.c(), recipe=recipe.c(),
                  defer_update=int(defer_update), dh_debug=_ptr(g.dh_debug), gemm_ws=_ptr(g.gemm_ws),
                  gemm_ws_bytes=g.gemm_ws.numel() if g.gemm_ws is not None else 0)
    _check(_c_mlp_bwd(C.byref(a), _stream(stream)))
    return g


# ------------------------------------------------------------------ 16- and 32-bit operators
_ELEM = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ACTS = {"none": 0, "gelu": 1, "relu": 2, "silu": 3}
_NO_CKPT = CCkpt(None, None, 0)


def _elem(t, name, kinds=_ELEM) -> int:
    e = kinds.get(t.dtype)
    if e is None:
        raise TypeError(f"{name} is {t.dtype}: expected one of {', '.join(str(k) for k in kinds)}")
    return e


def _act(act) -> int:
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
    return ACTS[act]


def _where(t, name) -> None:
    """Says why a tensor is not on the current CUDA device."""
    if not t.is_cuda:
        raise TypeError(f"{name} is not a CUDA tensor")
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _dev(t, name) -> int:
    """The index of the current CUDA device, on which the tensor must be."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _where(t, name)
    return dev


def _rows(t, name, rows, cols, dtype, dev) -> int:
    """Checks a [rows, cols] tensor whose rows are contiguous; returns its row stride."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}: expected ({rows}, {cols})")
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}: expected {dtype}")
    if t.get_device() != dev:
        _where(t, name)
    if t.is_contiguous():
        return cols
    s0, s1 = t.stride()
    if (cols > 1 and s1 != 1) or (rows > 1 and s0 < cols):
        raise ValueError(f"{name} has strides {(s0, s1)}: rows must be contiguous and not overlap")
    return s0 if rows > 1 else cols


def _flat(t, name, shape, dtype, dev) -> None:
    """Checks a contiguous tensor of the given shape and type."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}: expected {shape}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}: expected {dtype}")
    if t.get_device() != dev:
        _where(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")


def _given_ws(t, dev):
    """Checks a workspace that the caller keeps (all of its bytes there: contiguous)."""
    if t.get_device() != dev:
        _where(t, "grads.workspace")
    if not t.is_contiguous():
        raise ValueError("grads.workspace is not contiguous")
    return t


# The current stream's handle without the Stream object around it (4 us less per call where
# this PyTorch offers it).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on(stream, dev):
    """Context in which a call runs on a given stream: what it allocates belongs to that stream."""
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
    return torch.cuda.stream(stream)


@dataclass
class ActCkpt:
    """An 8-bit checkpoint of a [rows, cols] tensor: FP8 codes [rows, cols] uint8 and, per 32
    columns of a row, a scale byte b (value = code * 2^(b - 127)) in scales [rows, 4 ceil(cols / 128)]."""
    codes: torch.Tensor
    scales: torch.Tensor
    dtype: int = E4M3

    @property
    def shape(self):
        return self.codes.shape

    def c(self, rows, cols, dev, name="ckpt") -> CCkpt:
        _flat(self.codes, name + ".codes", (rows, cols), torch.uint8, dev)
        _flat(self.scales, name + ".scales", (rows, (cols + 127) // 128 * 4), torch.uint8, dev)
        return CCkpt(self.codes.data_ptr(), self.scales.data_ptr(), self.dtype)


def act_ckpt_scale_pitch(cols) -> int:
    return int(_c_ckpt_pitch(cols))


def _new_ckpt(rows, cols, dtype, device):
    """A checkpoint and its C form (nothing in it to check)."""
    codes, scales = _e((rows, cols), torch.uint8, device), _e((rows, (cols + 127) // 128 * 4), torch.uint8, device)
    return ActCkpt(codes, scales, dtype), CCkpt(codes.data_ptr(), scales.data_ptr(), dtype)


def act_ckpt(rows, cols, *, dtype=E4M3, device="cuda") -> ActCkpt:
    """An uninitialised checkpoint of a [rows, cols] tensor."""
    return ActCkpt(_e((rows, cols), torch.uint8, device), _e((rows, (cols + 127) // 128 * 4), torch.uint8, device), dtype)


def act_ckpt_save(x, *, dtype=E4M3, ckpt: ActCkpt | None = None, stream=None) -> ActCkpt:
    """Saves a 2-D bf16, fp16 or fp32 tensor as an 8-bit checkpoint (into `ckpt` if given, in its format)."""
    elem = _elem(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}: expected two dimensions")
    rows, cols = x.shape
    dev = _dev(x, "x")
    if stream is not None:
        with _on(stream, dev):
            return act_ckpt_save(x, dtype=dtype, ckpt=ckpt)
    ldx = _rows(x, "x", rows, cols, x.dtype, dev)
    if ckpt is None:
        ckpt, cc = _new_ckpt(rows, cols, dtype, x.device)
    else:
        cc = ckpt.c(rows, cols, dev)
    _check(_c_ckpt_save(x.data_ptr(), elem, rows, cols, ldx, C.byref(cc), _raw_stream(dev)))
    return ckpt


def act_ckpt_restore(ckpt: ActCkpt, *, out_dtype=torch.bfloat16, act="none", gamma=None, beta=None, out=None,
                     stream=None) -> torch.Tensor:
    """The checkpoint's values, or act(values), or values * gamma + beta per column (a LayerNorm's
    output from its checkpointed rows). Values beyond the type's range saturate."""
    rows, cols = ckpt.codes.shape
    dev = _dev(ckpt.codes, "ckpt.codes")
    if stream is not None:
        with _on(stream, dev):
            return act_ckpt_restore(ckpt, out_dtype=out_dtype, act=act, gamma=gamma, beta=beta, out=out)
    cc = ckpt.c(rows, cols, dev)
    pe = 0
    if gamma is not None and beta is not None:
        pe = _elem(gamma, "gamma")
        _flat(gamma, "gamma", (cols,), gamma.dtype, dev)
        _flat(beta, "beta", (cols,), gamma.dtype, dev)
    ldo = cols
    if out is None:
        out = _e((rows, cols), out_dtype, ckpt.codes.device)
    else:
        ldo = _rows(out, "out", rows, cols, out.dtype, dev)
    _check(_c_ckpt_restore(C.byref(cc), rows, cols, _act(act), _ptr(gamma), _ptr(beta), pe, out.data_ptr(),
                           _elem(out, "out"), ldo, _raw_stream(dev)))
    return out


@dataclass
class LayerNormCtx:
    """What a LayerNorm's backward needs: rsigma, and the normalised input x (the sum, after a
    fused residual) with mu, or the checkpoint of the normalised rows."""
    x: torch.Tensor | None
    mu: torch.Tensor | None
    rsigma: torch.Tensor
    ckpt: ActCkpt | None = None


def layernorm_fwd(x, gamma, beta, *, eps=1e-5, residual=None, ckpt=False, y=None, stream=None):
    """LayerNorm of a 2-D bf16, fp16 or fp32 tensor, output of the same type; returns (y, ctx).
    gamma and beta are of one type, any of the three. residual: h = x + residual (rounded to the
    type) is normalised and returned as ctx.x. ckpt: True (E4M3) or an ActCkpt to fill; the
    normalised rows are kept in 8 bits and the backward reads those, so x may be dropped."""
    elem, pe = _elem(x, "x"), _elem(gamma, "gamma")
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}: expected two dimensions")
    M, D = x.shape
    dt, dev, device = x.dtype, _dev(x, "x"), x.device
    if stream is not None:
        with _on(stream, dev):
            return layernorm_fwd(x, gamma, beta, eps=eps, residual=residual, ckpt=ckpt, y=y)
    ldx = _rows(x, "x", M, D, dt, dev)
    _flat(gamma, "gamma", (D,), gamma.dtype, dev)
    _flat(beta, "beta", (D,), gamma.dtype, dev)
    ldr = _rows(residual, "residual", M, D, dt, dev) if residual is not None else 0
    ldy = D
    if y is None:
        y = _e((M, D), dt, device)
    else:
        ldy = _rows(y, "y", M, D, dt, dev)
    mu, rs = _e((M,), torch.float32, device), _e((M,), torch.float32, device)
    h, hp = x, None
    if residual is not None:
        h = _e((M, D), dt, device)
        hp = h.data_ptr()
    if ckpt is False or ckpt is None:
        ckpt, cc = None, _NO_CKPT
    elif ckpt is True:
        ckpt, cc = _new_ckpt(M, D, E4M3, device)
    else:
        cc = ckpt.c(M, D, dev)
    a = CLayerNormFwd(M, D, elem, pe, x.data_ptr(), _ptr(residual), gamma.data_ptr(), beta.data_ptr(), y.data_ptr(), hp,
                      mu.data_ptr(), rs.data_ptr(), cc, ldx, ldr, ldy, eps)
    _check(_c_layernorm_fwd(C.byref(a), _raw_stream(dev)))
    return y, LayerNormCtx(h, mu, rs, ckpt)


@dataclass
class LayerNormGrads:
    """Gradients of layernorm_bwd. workspace: scratch that the caller keeps from call to call; None: each call takes
    its own from the current stream's memory and gives it back."""
    dx: torch.Tensor
    dgamma: torch.Tensor
    dbeta: torch.Tensor
    workspace: torch.Tensor | None = None


def layernorm_bwd_workspace_size(M, D) -> int:
    return int(_c_layernorm_bwd_ws(M, D))


def _layernorm_ws(M, D, device):
    return _e((_c_layernorm_bwd_ws(M, D),), torch.uint8, device)


def layernorm_grads(M, D, *, dtype=torch.bfloat16, device="cuda", workspace=True) -> LayerNormGrads:
    """Gradients of one layernorm_bwd, with a workspace to keep."""
    return LayerNormGrads(_e((M, D), dtype, device), _e((D,), torch.float32, device), _e((D,), torch.float32, device),
                          _layernorm_ws(M, D, device) if workspace else None)


def layernorm_bwd(dy, ctx: LayerNormCtx, gamma, *, dresidual=None, grads: LayerNormGrads | None = None,
                  stream=None) -> LayerNormGrads:
    """Gradients of layernorm_fwd: dx (plus dresidual, the residual stream's own gradient), and
    dgamma, dbeta in fp32 (summed in a fixed order). Reads ctx.ckpt if there is one, else ctx.x."""
    elem, pe = _elem(dy, "dy"), _elem(gamma, "gamma")
    if dy.dim() != 2:
        raise ValueError(f"dy has shape {tuple(dy.shape)}: expected two dimensions")
    M, D = dy.shape
    dt, dev = dy.dtype, _dev(dy, "dy")
    if stream is not None:
        with _on(stream, dev):
            return layernorm_bwd(dy, ctx, gamma, dresidual=dresidual, grads=grads)
    lddy = _rows(dy, "dy", M, D, dt, dev)
    _flat(gamma, "gamma", (D,), gamma.dtype, dev)
    _flat(ctx.rsigma, "ctx.rsigma", (M,), torch.float32, dev)
    if ctx.ckpt is not None:
        ck, x, mu, ldx = ctx.ckpt.c(M, D, dev), None, None, 0
    elif ctx.x is None or ctx.mu is None:
        raise ValueError("ctx holds neither a checkpoint nor x and mu")
    else:
        ck, x, mu = _NO_CKPT, ctx.x.data_ptr(), ctx.mu.data_ptr()
        ldx = _rows(ctx.x, "ctx.x", M, D, dt, dev)
        _flat(ctx.mu, "ctx.mu", (M,), torch.float32, dev)
    lddr = _rows(dresidual, "dresidual", M, D, dt, dev) if dresidual is not None else 0
    lddx = D
    if grads is None:
        grads = layernorm_grads(M, D, dtype=dt, device=dy.device, workspace=False)
    else:
        lddx = _rows(grads.dx, "grads.dx", M, D, dt, dev)
        _flat(grads.dgamma, "grads.dgamma", (D,), torch.float32, dev)
        _flat(grads.dbeta, "grads.dbeta", (D,), torch.float32, dev)
    ws = _layernorm_ws(M, D, dy.device) if grads.workspace is None else _given_ws(grads.workspace, dev)
    a = CLayerNormBwd(M, D, elem, pe, dy.data_ptr(), x, mu, ctx.rsigma.data_ptr(), ck, gamma.data_ptr(), _ptr(dresidual),
                      grads.dx.data_ptr(), grads.dgamma.data_ptr(), grads.dbeta.data_ptr(), ws.data_ptr(), ws.nbytes, lddy,
                      ldx, lddr, lddx)
    _check(_c_layernorm_bwd(C.byref(a), _raw_stream(dev)))
    return grads


_ELEM16 = {torch.bfloat16: 0, torch.float16: 1}


@dataclass
class LinearActCtx:
    """What linear_act_bwd needs of its forward besides x and w: the activation and the
    pre-activation, as a tensor or as a checkpoint (neither for act "none")."""
    act: str = "none"
    h: torch.Tensor | None = None
    ckpt: ActCkpt | None = None


def linear_act_fwd(x, w, bias=None, *, act="none", residual=None, save="none", y=None, ctx: LinearActCtx | None = None,
                   stream=None):
    """act(x w^T + bias) + residual of bf16 or fp16 tensors, x [M, K], w [N, K]; returns (y, ctx).
    act: "none", "gelu" (tanh form), "relu" or "silu". save: what the backward reads of the
    pre-activation, "h" (a tensor), "ckpt" (8 bits) or "none"; the buffers of `ctx` are used if it has them."""
    elem, ia = _elem(x, "x", _ELEM16), _act(act)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError(f"x and w have shapes {tuple(x.shape)} and {tuple(w.shape)}: expected two dimensions")
    if save not in ("none", "h", "ckpt"):
        raise ValueError(f"unknown save {save!r}: one of none, h, ckpt")
    M, K = x.shape
    N = w.shape[0]
    dt, dev = x.dtype, _dev(x, "x")
    if stream is not None:
        with _on(stream, dev):
            return linear_act_fwd(x, w, bias, act=act, residual=residual, save=save, y=y, ctx=ctx)
    ldx = _rows(x, "x", M, K, dt, dev)
    _flat(w, "w", (N, K), dt, dev)
    if bias is not None:
        _flat(bias, "bias", (N,), dt, dev)
    ldr = _rows(residual, "residual", M, N, dt, dev) if residual is not None else 0
    ldy = N
    if y is None:
        y = _e((M, N), dt, x.device)
    else:
        ldy = _rows(y, "y", M, N, dt, dev)
    if ctx is None:
        ctx = LinearActCtx()
    ctx.act = act
    h, ck = None, _NO_CKPT
    if save == "h":
        ctx.ckpt = None
        if ctx.h is None:
            ctx.h = _e((M, N), dt, x.device)
        else:
            _flat(ctx.h, "ctx.h", (M, N), dt, dev)
        h = ctx.h.data_ptr()
    elif save == "ckpt":
        ctx.h = None
        if ctx.ckpt is None:
            ctx.ckpt, ck = _new_ckpt(M, N, E4M3, x.device)
        else:
            ck = ctx.ckpt.c(M, N, dev, "ctx.ckpt")
    else:
        ctx.h = ctx.ckpt = None
    a = CLinearActFwd(M, K, N, elem, ia, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), h, ck, ldx,
                      ldr, ldy)
    _check(_c_linear_act_fwd(C.byref(a), _raw_stream(dev)))
    return y, ctx


@dataclass
class LinearActGrads:
    """Gradients of linear_act_bwd. workspace: scratch (dz and a restored x, most of it) that the caller keeps from call
    to call; None: each call takes its own from the current stream's memory and gives it back."""
    dx: torch.Tensor | None
    dw: torch.Tensor | None
    dbias: torch.Tensor | None
    workspace: torch.Tensor | None = None


def linear_act_bwd_workspace_size(M, K, N, *, has_act, x_from_ckpt) -> int:
    return int(_c_linear_act_bwd_ws(M, K, N, int(has_act), int(x_from_ckpt)))


def _linear_act_ws(M, K, N, act, x_from_ckpt, device):
    return _e((_c_linear_act_bwd_ws(M, K, N, int(act != "none"), int(x_from_ckpt)),), torch.uint8, device)


def linear_act_grads(M, K, N, *, act="none", x_from_ckpt=False, dx=True, dw=True, bias=True, dtype=torch.bfloat16,
                     device="cuda", workspace=True) -> LinearActGrads:
    """Gradients of one linear_act_bwd, with a workspace to keep; dx, dw, bias=False leave theirs out."""
    return LinearActGrads(_e((M, K), dtype, device) if dx else None, _e((N, K), dtype, device) if dw else None,
                          _e((N,), torch.float32, device) if bias else None,
                          _linear_act_ws(M, K, N, act, x_from_ckpt, device) if workspace else None)


def linear_act_bwd(dy, x, w, ctx: LinearActCtx, *, x_act="none", x_gamma=None, x_beta=None,
                   grads: LinearActGrads | None = None, stream=None) -> LinearActGrads:
    """Gradients of linear_act_fwd (the residual's is dy). x: the forward's input, or an ActCkpt from
    which it is restored as x_act(values) or values * x_gamma + x_beta. Gradients that `grads` leaves
    None are not computed; x may be None without dw."""
    elem, ia = _elem(dy, "dy", _ELEM16), _act(ctx.act)
    if dy.dim() != 2 or w.dim() != 2:
        raise ValueError(f"dy and w have shapes {tuple(dy.shape)} and {tuple(w.shape)}: expected two dimensions")
    M, N = dy.shape
    K = w.shape[1]
    dt, dev = dy.dtype, _dev(dy, "dy")
    if stream is not None:
        with _on(stream, dev):
            return linear_act_bwd(dy, x, w, ctx, x_act=x_act, x_gamma=x_gamma, x_beta=x_beta, grads=grads)
    lddy = _rows(dy, "dy", M, N, dt, dev)
    _flat(w, "w", (N, K), dt, dev)
    h, hck, xp, xck, ldx = None, _NO_CKPT, None, _NO_CKPT, 0
    if ia:
        if ctx.ckpt is not None:
            hck = ctx.ckpt.c(M, N, dev, "ctx.ckpt")
        elif ctx.h is not None:
            _flat(ctx.h, "ctx.h", (M, N), dt, dev)
            h = ctx.h.data_ptr()
        else:
            raise ValueError(f"the forward with act {ctx.act!r} saved no pre-activation")
    if isinstance(x, ActCkpt):
        xck = x.c(M, K, dev, "x")
    elif x is not None:
        ldx = _rows(x, "x", M, K, dt, dev)
        xp = x.data_ptr()
    if x_gamma is not None:
        _flat(x_gamma, "x_gamma", (K,), dt, dev)
    if x_beta is not None:
        _flat(x_beta, "x_beta", (K,), dt, dev)
    lddx = K
    if grads is None:
        grads = linear_act_grads(M, K, N, dw=x is not None, dtype=dt, device=dy.device, workspace=False)
    else:
        if grads.dx is not None:
            lddx = _rows(grads.dx, "grads.dx", M, K, dt, dev)
        if grads.dw is not None:
            _flat(grads.dw, "grads.dw", (N, K), dt, dev)
        if grads.dbias is not None:
            _flat(grads.dbias, "grads.dbias", (N,), torch.float32, dev)
    ws = grads.workspace
    ws = _linear_act_ws(M, K, N, ctx.act, xck is not _NO_CKPT, dy.device) if ws is None else _given_ws(ws, dev)
    a = CLinearActBwd(M, K, N, elem, ia, dy.data_ptr(), xp, xck, _act(x_act), _ptr(x_gamma), _ptr(x_beta), w.data_ptr(), h,
                      hck, _ptr(grads.dx), _ptr(grads.dw), _ptr(grads.dbias), ws.data_ptr(), ws.nbytes, lddy, ldx, lddx)
    _check(_c_linear_act_bwd(C.byref(a), _raw_stream(dev)))
    return grads
