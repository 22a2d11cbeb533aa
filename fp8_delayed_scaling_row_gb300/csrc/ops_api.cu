// C ABI of the 16/32-bit operators: layernorm_fwd / layernorm_bwd, act_ckpt_save /
// act_ckpt_restore and linear_act_fwd / linear_act_bwd. Checks every argument
// before anything is enqueued, fills in the default row strides, and runs the
// launchers of layernorm_rows.cu, act_ckpt.cu and linear.cu.
#include "common.cuh"
#include "internal.h"

using namespace lnfp8;

namespace {

#define TRY(x)                             \
  do {                                     \
    const lnfp8_status _s = (x);           \
    if (_s != LNFP8_OK) return _s;         \
  } while (0)

constexpr int64_t kMaxRows = (1ll << 31) - 1;
constexpr int64_t kMaxTokens = (1ll << 31) - 1024;  // linear_act: tile rows past the last token stay 32-bit numbers
constexpr int64_t kMaxCols = 1ll << 30;
constexpr int64_t kMaxFeature = (1ll << 30) - 32;  // linear_act: two column sums of each, rounded up to 32, are counted in 32 bits

int elem_size(int elem) { return elem == LNFP8_FP32 ? 4 : 2; }

lnfp8_status need(const void* p, int align, const char* name, const char* who) {
  if (!p) return set_error(LNFP8_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
  if (reinterpret_cast<uintptr_t>(p) % align)
    return set_error(LNFP8_ERR_INVALID_ARG, "%s: %s is not %d-byte aligned", who, name, align);
  return LNFP8_OK;
}
lnfp8_status maybe(const void* p, int align, const char* name, const char* who) {
  return p ? need(p, align, name, who) : LNFP8_OK;
}

lnfp8_status check_elem(int e, const char* name, const char* who) {
  if (e < LNFP8_BF16 || e > LNFP8_FP32) return set_error(LNFP8_ERR_INVALID_ARG, "%s: bad %s %d", who, name, e);
  return LNFP8_OK;
}
lnfp8_status check_elem16(int e, const char* who) {
  if (e != LNFP8_BF16 && e != LNFP8_FP16) return set_error(LNFP8_ERR_INVALID_ARG, "%s: elem %d (bf16 or fp16)", who, e);
  return LNFP8_OK;
}
lnfp8_status check_act(int act, const char* name, const char* who) {
  if (act < LNFP8_ACT_NONE || act > LNFP8_ACT_SILU) return set_error(LNFP8_ERR_INVALID_ARG, "%s: bad %s %d", who, name, act);
  return LNFP8_OK;
}
lnfp8_status check_rows(int64_t v, const char* name, const char* who, int64_t most = kMaxRows) {
  if (v < 0) return set_error(LNFP8_ERR_INVALID_ARG, "%s: %s = %lld < 0", who, name, (long long)v);
  if (v > most) return set_error(LNFP8_ERR_UNSUPPORTED_SHAPE, "%s: %s = %lld too large", who, name, (long long)v);
  return LNFP8_OK;
}
lnfp8_status check_cols(int64_t v, int64_t most, const char* name, const char* who) {
  if (v < 1 || v > most)
    return set_error(LNFP8_ERR_UNSUPPORTED_SHAPE, "%s: %s = %lld must be 1..%lld", who, name, (long long)v, (long long)most);
  return LNFP8_OK;
}
// 0 means contiguous; anything else is at least the row's width.
lnfp8_status fill_ld(int64_t* ld, int64_t cols, const char* name, const char* who) {
  if (*ld == 0) *ld = cols;
  if (*ld < cols || *ld > (1ll << 40))
    return set_error(LNFP8_ERR_INVALID_ARG, "%s: %s = %lld, rows have %lld columns", who, name, (long long)*ld, (long long)cols);
  return LNFP8_OK;
}
// Feature sizes and row strides of the tensor-core products: 16-byte rows.
lnfp8_status check_feature(int64_t v, const char* name, const char* who) {
  if (v < 8 || v % 8 != 0 || v > kMaxFeature)
    return set_error(LNFP8_ERR_UNSUPPORTED_SHAPE, "%s: %s = %lld must be a positive multiple of 8 up to %lld", who, name, (long long)v,
                     (long long)kMaxFeature);
  return LNFP8_OK;
}
lnfp8_status fill_ld8(int64_t* ld, int64_t cols, const char* name, const char* who) {
  TRY(fill_ld(ld, cols, name, who));
  if (*ld % 8 != 0) return set_error(LNFP8_ERR_INVALID_ARG, "%s: %s = %lld is not a multiple of 8", who, name, (long long)*ld);
  return LNFP8_OK;
}
lnfp8_status check_ckpt(const lnfp8_ckpt& c, int code_align, const char* name, const char* who) {
  if (c.dtype != LNFP8_E4M3 && c.dtype != LNFP8_E5M2)
    return set_error(LNFP8_ERR_INVALID_ARG, "%s: bad FP8 dtype %d of %s", who, c.dtype, name);
  TRY(need(c.codes, code_align, name, who));
  return need(c.scales, 4, name, who);
}

}  // namespace

extern "C" {

int64_t lnfp8_act_ckpt_scale_pitch(int64_t cols) { return cols < 0 ? -1 : (cols + 127) / 128 * 4; }

lnfp8_status act_ckpt_save(const void* x, int elem, int64_t rows, int64_t cols, int64_t ldx, const lnfp8_ckpt* ckpt,
                           lnfp8_stream stream) {
  const char* who = "act_ckpt_save";
  clear_error();
  TRY(check_elem(elem, "elem", who));
  TRY(check_rows(rows, "rows", who));
  TRY(check_cols(cols, kMaxCols, "cols", who));
  TRY(fill_ld(&ldx, cols, "ldx", who));
  if (!ckpt) return set_error(LNFP8_ERR_INVALID_ARG, "%s: ckpt is NULL", who);
  if (rows > 0) {
    TRY(need(x, elem_size(elem), "x", who));
    TRY(check_ckpt(*ckpt, 1, "ckpt", who));
  }
  return act_ckpt_save_launch(x, elem, rows, cols, ldx, *ckpt, (cudaStream_t)stream);
}

lnfp8_status act_ckpt_restore(const lnfp8_ckpt* ckpt, int64_t rows, int64_t cols, int act, const void* gamma,
                              const void* beta, int param_elem, void* out, int elem, int64_t ldo, lnfp8_stream stream) {
  const char* who = "act_ckpt_restore";
  clear_error();
  TRY(check_elem(elem, "elem", who));
  TRY(check_act(act, "act", who));
  TRY(check_rows(rows, "rows", who));
  TRY(check_cols(cols, kMaxCols, "cols", who));
  TRY(fill_ld(&ldo, cols, "ldo", who));
  if (!ckpt) return set_error(LNFP8_ERR_INVALID_ARG, "%s: ckpt is NULL", who);
  if ((gamma == nullptr) != (beta == nullptr))
    return set_error(LNFP8_ERR_INVALID_ARG, "%s: gamma and beta come together", who);
  if (gamma) {
    if (act != LNFP8_ACT_NONE) return set_error(LNFP8_ERR_UNSUPPORTED, "%s: an activation and gamma, beta in one call", who);
    TRY(check_elem(param_elem, "param_elem", who));
    TRY(need(gamma, elem_size(param_elem), "gamma", who));
    TRY(need(beta, elem_size(param_elem), "beta", who));
  }
  if (rows > 0) {
    TRY(need(out, elem_size(elem), "out", who));
    TRY(check_ckpt(*ckpt, 1, "ckpt", who));
  }
  return act_ckpt_restore_launch(*ckpt, rows, cols, act, gamma, beta, param_elem, out, elem, ldo, (cudaStream_t)stream);
}

lnfp8_status layernorm_fwd(const lnfp8_layernorm_fwd_args* args, lnfp8_stream stream) {
  const char* who = "layernorm_fwd";
  clear_error();
  if (!args) return set_error(LNFP8_ERR_INVALID_ARG, "%s: args is NULL", who);
  lnfp8_layernorm_fwd_args a = *args;
  TRY(check_elem(a.elem, "elem", who));
  TRY(check_elem(a.param_elem, "param_elem", who));
  TRY(check_rows(a.M, "M", who));
  TRY(check_cols(a.D, layernorm_max_d(), "D", who));
  TRY(fill_ld(&a.ldx, a.D, "ldx", who));
  TRY(fill_ld(&a.ld_residual, a.D, "ld_residual", who));
  TRY(fill_ld(&a.ldy, a.D, "ldy", who));
  if (!(a.eps >= 0.f)) return set_error(LNFP8_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  const int es = elem_size(a.elem), ps = elem_size(a.param_elem);
  TRY(need(a.gamma, ps, "gamma", who));
  TRY(need(a.beta, ps, "beta", who));
  if (a.M > 0) {
    TRY(need(a.x, es, "x", who));
    TRY(need(a.y, es, "y", who));
    TRY(need(a.mu, 4, "mu", who));
    TRY(need(a.rsigma, 4, "rsigma", who));
    if (a.residual) {
      TRY(need(a.residual, es, "residual", who));
      TRY(need(a.x_sum, es, "x_sum", who));
    }
    if (a.ckpt.codes || a.ckpt.scales) TRY(check_ckpt(a.ckpt, 1, "ckpt", who));
  }
  return layernorm_fwd_launch(&a, (cudaStream_t)stream);
}

int64_t lnfp8_layernorm_bwd_workspace_size(int64_t M, int64_t D) {
  return M < 0 || D < 0 ? -1 : layernorm_bwd_ws_bytes(M, D);
}

lnfp8_status layernorm_bwd(const lnfp8_layernorm_bwd_args* args, lnfp8_stream stream) {
  const char* who = "layernorm_bwd";
  clear_error();
  if (!args) return set_error(LNFP8_ERR_INVALID_ARG, "%s: args is NULL", who);
  lnfp8_layernorm_bwd_args a = *args;
  TRY(check_elem(a.elem, "elem", who));
  TRY(check_elem(a.param_elem, "param_elem", who));
  TRY(check_rows(a.M, "M", who));
  TRY(check_cols(a.D, layernorm_max_d(), "D", who));
  TRY(fill_ld(&a.ld_dy, a.D, "ld_dy", who));
  TRY(fill_ld(&a.ldx, a.D, "ldx", who));
  TRY(fill_ld(&a.ld_dresidual, a.D, "ld_dresidual", who));
  TRY(fill_ld(&a.ld_dx, a.D, "ld_dx", who));
  const int es = elem_size(a.elem);
  TRY(need(a.gamma, elem_size(a.param_elem), "gamma", who));
  TRY(need(a.dgamma, 4, "dgamma", who));
  TRY(need(a.dbeta, 4, "dbeta", who));
  if (a.M > 0) {
    TRY(need(a.dy, es, "dy", who));
    TRY(need(a.dx, es, "dx", who));
    TRY(need(a.rsigma, 4, "rsigma", who));
    if (a.ckpt.codes || a.ckpt.scales) {
      TRY(check_ckpt(a.ckpt, 1, "ckpt", who));
      if (a.x) return set_error(LNFP8_ERR_INVALID_ARG, "%s: x and a checkpoint", who);
    } else {
      TRY(need(a.x, es, "x", who));
      TRY(need(a.mu, 4, "mu", who));
    }
    TRY(maybe(a.dresidual, es, "dresidual", who));
    TRY(need(a.workspace, 16, "workspace", who));
    if (a.workspace_bytes < layernorm_bwd_ws_bytes(a.M, a.D))
      return set_error(LNFP8_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who, (long long)a.workspace_bytes,
                       (long long)layernorm_bwd_ws_bytes(a.M, a.D));
  }
  return layernorm_bwd_launch(&a, (cudaStream_t)stream);
}

lnfp8_status linear_act_fwd(const lnfp8_linear_act_fwd_args* args, lnfp8_stream stream) {
  const char* who = "linear_act_fwd";
  clear_error();
  if (!args) return set_error(LNFP8_ERR_INVALID_ARG, "%s: args is NULL", who);
  lnfp8_linear_act_fwd_args a = *args;
  TRY(check_elem16(a.elem, who));
  TRY(check_act(a.act, "act", who));
  TRY(check_rows(a.M, "M", who, kMaxTokens));
  TRY(check_feature(a.K, "K", who));
  TRY(check_feature(a.N, "N", who));
  TRY(fill_ld8(&a.ldx, a.K, "ldx", who));
  TRY(fill_ld8(&a.ld_residual, a.N, "ld_residual", who));
  TRY(fill_ld8(&a.ldy, a.N, "ldy", who));
  TRY(need(a.w, 16, "w", who));
  TRY(maybe(a.bias, 16, "bias", who));
  if (a.M > 0) {
    TRY(need(a.x, 16, "x", who));
    TRY(need(a.y, 16, "y", who));
    TRY(maybe(a.residual, 16, "residual", who));
    TRY(maybe(a.h, 16, "h", who));
    if (a.ckpt.codes || a.ckpt.scales) {
      TRY(check_ckpt(a.ckpt, 8, "ckpt", who));
      if (a.h) return set_error(LNFP8_ERR_INVALID_ARG, "%s: h and a checkpoint", who);
    }
  }
  return linear_act_fwd_launch(&a, (cudaStream_t)stream);
}

int64_t lnfp8_linear_act_bwd_workspace_size(int64_t M, int64_t K, int64_t N, int has_act, int x_from_ckpt) {
  return M < 0 || K < 0 || N < 0 ? -1 : linear_act_bwd_ws_bytes(M, K, N, has_act != 0, x_from_ckpt != 0);
}

lnfp8_status linear_act_bwd(const lnfp8_linear_act_bwd_args* args, lnfp8_stream stream) {
  const char* who = "linear_act_bwd";
  clear_error();
  if (!args) return set_error(LNFP8_ERR_INVALID_ARG, "%s: args is NULL", who);
  lnfp8_linear_act_bwd_args a = *args;
  TRY(check_elem16(a.elem, who));
  TRY(check_act(a.act, "act", who));
  TRY(check_act(a.x_act, "x_act", who));
  TRY(check_rows(a.M, "M", who, kMaxTokens));
  TRY(check_feature(a.K, "K", who));
  TRY(check_feature(a.N, "N", who));
  TRY(fill_ld8(&a.ld_dy, a.N, "ld_dy", who));
  TRY(fill_ld8(&a.ldx, a.K, "ldx", who));
  TRY(fill_ld8(&a.ld_dx, a.K, "ld_dx", who));
  TRY(maybe(a.dw, 16, "dw", who));
  TRY(maybe(a.dbias, 4, "dbias", who));
  const bool xck = a.x_ckpt.codes || a.x_ckpt.scales, hck = a.h_ckpt.codes || a.h_ckpt.scales;
  if (a.M > 0) {
    TRY(need(a.dy, 16, "dy", who));
    TRY(maybe(a.dx, 16, "dx", who));
    if (a.dx) TRY(need(a.w, 16, "w", who));
    if (a.act != LNFP8_ACT_NONE) {
      if (hck) {
        TRY(check_ckpt(a.h_ckpt, 8, "h_ckpt", who));
        if (a.h) return set_error(LNFP8_ERR_INVALID_ARG, "%s: h and a checkpoint of it", who);
      } else {
        TRY(need(a.h, 16, "h", who));
      }
    }
    if (a.dw) {
      if (xck) {
        TRY(check_ckpt(a.x_ckpt, 8, "x_ckpt", who));
        if (a.x) return set_error(LNFP8_ERR_INVALID_ARG, "%s: x and a checkpoint of x", who);
        if ((a.x_gamma == nullptr) != (a.x_beta == nullptr))
          return set_error(LNFP8_ERR_INVALID_ARG, "%s: x_gamma and x_beta come together", who);
        if (a.x_gamma && a.x_act != LNFP8_ACT_NONE)
          return set_error(LNFP8_ERR_UNSUPPORTED, "%s: x_act and x_gamma, x_beta in one call", who);
        TRY(maybe(a.x_gamma, 16, "x_gamma", who));
        TRY(maybe(a.x_beta, 16, "x_beta", who));
      } else {
        TRY(need(a.x, 16, "x", who));
        if (a.x_act != LNFP8_ACT_NONE || a.x_gamma || a.x_beta)
          return set_error(LNFP8_ERR_INVALID_ARG, "%s: x_act, x_gamma, x_beta restore a checkpoint", who);
      }
    }
    const int64_t want = linear_act_bwd_ws_bytes(a.M, a.K, a.N, a.act != LNFP8_ACT_NONE, xck);
    if (want > 0) {
      TRY(need(a.workspace, 16, "workspace", who));
      if (a.workspace_bytes < want)
        return set_error(LNFP8_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who, (long long)a.workspace_bytes,
                         (long long)want);
    }
  }
  return linear_act_bwd_launch(&a, (cudaStream_t)stream);
}

}  // extern "C"
