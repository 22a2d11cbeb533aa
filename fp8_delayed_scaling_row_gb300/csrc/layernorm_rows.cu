// LayerNorm forward and backward with 16- or 32-bit output: the LayerNorms of a
// model that stay outside the FP8 modules (te.LayerNorm; TE tutorial, code block 1
// module tour, code block 2 MiniGPT's final norm). The forward can add a residual
// in front and keep its normalised rows xhat as an 8-bit checkpoint; the backward
// reads either the input with its statistics or that checkpoint.
//   forward   h = T(x + r), mu = mean(h), rs = 1/sqrt(mean((h - mu)^2) + eps),
//             xhat = (h - mu) rs, y = T(xhat gamma + beta)
//   backward  g = dy gamma, dx = T(rs (g - mean(g) - xhat mean(g xhat)) + dres),
//             dgamma = sum_rows dy xhat, dbeta = sum_rows dy
// All arithmetic is fp32; the statistics are two sums over the row in registers
// (the mean first, then the centred squares, so a large mean loses nothing).
#include "common.cuh"
#include "internal.h"
#include "rowmath.cuh"

namespace lnfp8 {
namespace {

constexpr int kMaxD = 16384;

// Sum over the TPR threads of a row group; every thread gets the result. `xch`
// holds two buffers of 32 floats per group, used in turn (`turn` counts the sums),
// so that one barrier per sum is enough.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* xch, int& turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  if constexpr (TPR == 32) {
    return make_float2(a, b);
  } else {
    constexpr int W = TPR / 32;
    const int group = threadIdx.x / TPR, w = (threadIdx.x % TPR) / 32, lane = threadIdx.x & 31;
    float2* buf = xch + (group * 2 + (turn++ & 1)) * W;
    if (lane == 0) buf[w] = make_float2(a, b);
    if constexpr (TPR == 1024) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(TPR) : "memory");
    if constexpr (W <= 8) {
      float sa = 0.f, sb = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        sa += buf[i].x;
        sb += buf[i].y;
      }
      return make_float2(sa, sb);
    } else {
      const float2 v = lane < W ? buf[lane] : make_float2(0.f, 0.f);
      return make_float2(warp_sum(v.x), warp_sum(v.y));
    }
  }
}

struct LnFwdParams {
  const void* x;
  const void* resid;
  const void* gamma;
  const void* beta;
  void* y;
  void* xsum;
  float* mu;
  float* rs;
  uint8_t* codes;
  uint8_t* scales;
  int64_t M, ldx, ldr, ldy, pitch;
  int D, param_elem;
  float eps;
};

struct LnBwdParams {
  const void* dy;
  const void* x;
  const float* mu;
  const float* rs;
  const uint8_t* codes;
  const uint8_t* scales;
  const void* gamma;
  const void* dres;
  void* dx;
  float* part;  // [blocks][2][D] column partials
  int64_t M, lddy, ldx, lddres, lddx, pitch;
  int D, param_elem;
};

// ------------------------------------------------------------ any width, any alignment
// A group of TPR threads owns a row; thread t holds columns t, t + TPR, ... (so that
// a warp reads 32 neighbours and a checkpoint block is one warp's value i).
template <int ELEM, int TPR, int NE, int CK>  // CK: -1 none, else the lnfp8_dtype of the codes
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
ln_fwd_any_kernel(const LnFwdParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int GPB = kThreads / TPR;
  __shared__ float2 xch[2 * kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const float inv_d = 1.0f / (float)p.D;
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * GPB; row0 < p.M; row0 += (int64_t)gridDim.x * GPB) {
    const int64_t row = row0 + g;
    const bool active = row < p.M;
    float v[NE];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = t + TPR * i;
      v[i] = 0.f;
      if (active && c < p.D) {
        v[i] = load_elem<ELEM>(p.x, row * p.ldx + c);
        if (p.resid) {
          v[i] = round_elem<ELEM>(v[i] + load_elem<ELEM>(p.resid, row * p.ldr + c));
          store_elem<ELEM>(p.xsum, row * p.D + c, v[i]);
        }
      }
      s += v[i];
    }
    const float mu = row_sum2<TPR>(s, 0.f, xch, turn).x * inv_d;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      v[i] -= mu;
      if (t + TPR * i < p.D) q = fmaf(v[i], v[i], q);
    }
    const float rs = 1.0f / sqrtf(row_sum2<TPR>(q, 0.f, xch, turn).x * inv_d + p.eps);
    if (!active) continue;  // uniform over the row group; the barriers above are behind it
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = t + TPR * i;
      const bool in = c < p.D;
      const float xh = v[i] * rs;
      if (in) {
        const float ga = load_elem_rt(p.gamma, p.param_elem, c), be = load_elem_rt(p.beta, p.param_elem, c);
        store_elem<ELEM>(p.y, row * p.ldy + c, fmaf(xh, ga, be));
      }
      if constexpr (CK >= 0) {
        const uint32_t b = ckpt_byte<CK>(warp_max_u32(in ? abs_bits(xh) : 0u));
        const uint16_t code = cvt_fp8x2<CK>(xh * ckpt_inv_scale(b), 0.f);
        if (in) p.codes[row * p.D + c] = (uint8_t)code;
        if ((threadIdx.x & 31) == 0 && in) p.scales[row * p.pitch + (c >> 5)] = (uint8_t)b;
      }
    }
    if (t == 0) {
      p.mu[row] = mu;
      p.rs[row] = rs;
    }
  }
}

template <int ELEM, int TPR, int NE, int CK>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
ln_bwd_any_kernel(const LnBwdParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int GPB = kThreads / TPR;
  __shared__ float2 xch[2 * kThreads / 32];
  extern __shared__ float colred[];  // [2][D], only with several row groups
  pdl_wait();
  pdl_launch_dependents();
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const float inv_d = 1.0f / (float)p.D;
  float accg[NE], accb[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) accg[i] = accb[i] = 0.f;
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * GPB; row0 < p.M; row0 += (int64_t)gridDim.x * GPB) {
    const int64_t row = row0 + g;
    const bool active = row < p.M;
    const float rs = active ? p.rs[row] : 0.f;
    const float mu = active && CK < 0 ? p.mu[row] : 0.f;
    float xh[NE], gg[NE];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = t + TPR * i;
      xh[i] = gg[i] = 0.f;
      if (active && c < p.D) {
        const float d = load_elem<ELEM>(p.dy, row * p.lddy + c);
        if constexpr (CK >= 0)
          xh[i] = fp8x2_to_f32<CK>(p.codes[row * p.D + c]).x * ckpt_scale(p.scales[row * p.pitch + (c >> 5)]);
        else
          xh[i] = (load_elem<ELEM>(p.x, row * p.ldx + c) - mu) * rs;
        accg[i] = fmaf(d, xh[i], accg[i]);
        accb[i] += d;
        gg[i] = d * load_elem_rt(p.gamma, p.param_elem, c);
      }
      s1 += gg[i];
      s2 = fmaf(gg[i], xh[i], s2);
    }
    const float2 sums = row_sum2<TPR>(s1, s2, xch, turn);
    if (!active) continue;  // uniform over the row group
    const float mg = sums.x * inv_d, mgx = sums.y * inv_d;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = t + TPR * i;
      if (c >= p.D) continue;
      float o = (fmaf(-mgx, xh[i], gg[i] - mg)) * rs;
      if (p.dres) o += load_elem<ELEM>(p.dres, row * p.lddres + c);
      store_elem<ELEM>(p.dx, row * p.lddx + c, o);
    }
  }
  // this block's column partials: the row groups add theirs in turn
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
  if constexpr (GPB > 1) {
    for (int turn_g = 0; turn_g < GPB; ++turn_g) {
      __syncthreads();
      if (g != turn_g) continue;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = t + TPR * i;
        if (c >= p.D) continue;
        colred[c] = turn_g ? colred[c] + accg[i] : accg[i];
        colred[p.D + c] = turn_g ? colred[p.D + c] + accb[i] : accb[i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.D; c += kThreads) part[c] = colred[c];
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = t + TPR * i;
      if (c >= p.D) continue;
      part[c] = accg[i];
      part[p.D + c] = accb[i];
    }
  }
}

// dst[c] = sum over n partial rows of part[i][c], c < cols, in a fixed order: 32 columns
// per block, 8 warps each adding every eighth row, then the warps' sums in order.
__global__ void __launch_bounds__(256) colsum_kernel(const float* __restrict__ part, int n, int cols, int split,
                                                     float* __restrict__ a, float* __restrict__ b) {
  __shared__ float red[8][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int i = w; i < n; i += 8) s += part[(int64_t)i * cols + c];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
    s = red[0][lane];
#pragma unroll
    for (int k = 1; k < 8; ++k) s += red[k][lane];
    if (c < split) a[c] = s;
    else b[c - split] = s;
  }
}

// Blocks of the backward's row pass: the partial rows it leaves are summed afterwards.
constexpr int kBwdBlocksPerSm = 2;

template <typename K>
lnfp8_status allow_smem(K kernel, size_t smem, const char* who) {
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return check_launch(who);
  return LNFP8_OK;
}

template <int ELEM, int CK>
lnfp8_status fwd_any(const LnFwdParams& p, cudaStream_t st) {
  auto go = [&](auto kernel, int tpr) {
    const int threads = tpr < 256 ? 256 : tpr, gpb = threads / tpr;
    const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * (2048 / threads));
    if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, p) != cudaSuccess) return check_launch("layernorm_fwd launch");
    return check_launch("layernorm_fwd");
  };
  if (p.D <= 512) return go(ln_fwd_any_kernel<ELEM, 32, 16, CK>, 32);
  if (p.D <= 2048) return go(ln_fwd_any_kernel<ELEM, 128, 16, CK>, 128);
  if (p.D <= 8192) return go(ln_fwd_any_kernel<ELEM, 512, 16, CK>, 512);
  return go(ln_fwd_any_kernel<ELEM, 1024, 16, CK>, 1024);
}

template <int ELEM, int CK>
lnfp8_status bwd_any(const LnBwdParams& p, int* blocks_out, cudaStream_t st) {
  auto go = [&](auto kernel, int tpr) {
    const int threads = tpr < 256 ? 256 : tpr, gpb = threads / tpr;
    const size_t smem = gpb > 1 ? 2 * (size_t)p.D * sizeof(float) : 0;
    const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * kBwdBlocksPerSm);
    *blocks_out = (int)blocks;
    if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), smem, st, p) != cudaSuccess) return check_launch("layernorm_bwd launch");
    return check_launch("layernorm_bwd");
  };
  if (p.D <= 512) return go(ln_bwd_any_kernel<ELEM, 32, 16, CK>, 32);
  if (p.D <= 2048) return go(ln_bwd_any_kernel<ELEM, 128, 16, CK>, 128);
  if (p.D <= 8192) return go(ln_bwd_any_kernel<ELEM, 512, 16, CK>, 512);
  return go(ln_bwd_any_kernel<ELEM, 1024, 16, CK>, 1024);
}

}  // namespace

int64_t layernorm_max_d() { return kMaxD; }

int64_t layernorm_bwd_ws_bytes(int64_t M, int64_t D) {
  if (M == 0) return 0;
  return min64(M, (int64_t)num_sms() * kBwdBlocksPerSm) * 2 * D * (int64_t)sizeof(float);
}

lnfp8_status colsum_launch(const float* part, int n, int cols, int split, float* a, float* b, cudaStream_t st) {
  LaunchScope ls("colsum", st);
  if (launch_pdl(colsum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, st, part, n, cols, split, a, b) != cudaSuccess)
    return check_launch("column sums launch");
  return check_launch("column sums");
}

#define BY_CKPT(ELEM, FN, ...)                                                                   \
  (ck < 0 ? FN<ELEM, -1>(__VA_ARGS__)                                                            \
          : ck == LNFP8_E4M3 ? FN<ELEM, LNFP8_E4M3>(__VA_ARGS__) : FN<ELEM, LNFP8_E5M2>(__VA_ARGS__))
#define BY_ELEM(FN, ...)                                                                         \
  (a->elem == LNFP8_BF16 ? BY_CKPT(LNFP8_BF16, FN, __VA_ARGS__)                                  \
                         : a->elem == LNFP8_FP16 ? BY_CKPT(LNFP8_FP16, FN, __VA_ARGS__) : BY_CKPT(LNFP8_FP32, FN, __VA_ARGS__))

lnfp8_status layernorm_fwd_launch(const lnfp8_layernorm_fwd_args* a, cudaStream_t st) {
  if (a->M == 0) return LNFP8_OK;
  LnFwdParams p;
  p.x = a->x;
  p.resid = a->residual;
  p.gamma = a->gamma;
  p.beta = a->beta;
  p.y = a->y;
  p.xsum = a->x_sum;
  p.mu = a->mu;
  p.rs = a->rsigma;
  p.codes = a->ckpt.codes;
  p.scales = a->ckpt.scales;
  p.M = a->M;
  p.ldx = a->ldx;
  p.ldr = a->ld_residual;
  p.ldy = a->ldy;
  p.pitch = lnfp8_act_ckpt_scale_pitch(a->D);
  p.D = (int)a->D;
  p.param_elem = a->param_elem;
  p.eps = a->eps;
  const int ck = a->ckpt.codes ? a->ckpt.dtype : -1;
  LaunchScope ls("layernorm_fwd", st);
  return BY_ELEM(fwd_any, p, st);
}

lnfp8_status layernorm_bwd_launch(const lnfp8_layernorm_bwd_args* a, cudaStream_t st) {
  if (a->M == 0) {
    if (cudaMemsetAsync(a->dgamma, 0, a->D * sizeof(float), st) != cudaSuccess ||
        cudaMemsetAsync(a->dbeta, 0, a->D * sizeof(float), st) != cudaSuccess)
      return check_launch("layernorm_bwd: clearing dgamma/dbeta");
    return LNFP8_OK;
  }
  LnBwdParams p;
  p.dy = a->dy;
  p.x = a->x;
  p.mu = a->mu;
  p.rs = a->rsigma;
  p.codes = a->ckpt.codes;
  p.scales = a->ckpt.scales;
  p.gamma = a->gamma;
  p.dres = a->dresidual;
  p.dx = a->dx;
  p.part = static_cast<float*>(a->workspace);
  p.M = a->M;
  p.lddy = a->ld_dy;
  p.ldx = a->ldx;
  p.lddres = a->ld_dresidual;
  p.lddx = a->ld_dx;
  p.pitch = lnfp8_act_ckpt_scale_pitch(a->D);
  p.D = (int)a->D;
  p.param_elem = a->param_elem;
  const int ck = a->ckpt.codes ? a->ckpt.dtype : -1;
  int blocks = 0;
  lnfp8_status s;
  {
    LaunchScope ls("layernorm_bwd", st);
    s = BY_ELEM(bwd_any, p, &blocks, st);
  }
  if (s != LNFP8_OK) return s;
  return colsum_launch(p.part, blocks, 2 * p.D, p.D, a->dgamma, a->dbeta, st);
}

}  // namespace lnfp8
