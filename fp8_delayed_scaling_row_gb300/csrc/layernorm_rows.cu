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

#include <algorithm>

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
  int D, param_elem, dt;  // dt: the lnfp8_dtype of the codes
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
  int D, param_elem, dt;
};

// ------------------------------------------------------------ any width, any alignment
// A group of TPR threads owns a row; thread t holds columns t, t + TPR, ... (so that
// a warp reads 32 neighbours and a checkpoint block is one warp's value i).
template <int ELEM, int TPR, int NE, bool CK>  // CK: with a checkpoint
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
      if constexpr (CK) {
        const uint32_t b = ckpt_byte(warp_max_u32(in ? abs_bits(xh) : 0u), p.dt);
        const uint32_t code = fp8x2(xh * ckpt_inv_scale(b), 0.f, p.dt);
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

template <int ELEM, int TPR, int NE, bool CK>
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
    const float mu = active && !CK ? p.mu[row] : 0.f;
    float xh[NE], gg[NE];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = t + TPR * i;
      xh[i] = gg[i] = 0.f;
      if (active && c < p.D) {
        const float d = load_elem<ELEM>(p.dy, row * p.lddy + c);
        if constexpr (CK)
          xh[i] = fp8x2_to_f32(p.codes[row * p.D + c], p.dt).x * ckpt_scale(p.scales[row * p.pitch + (c >> 5)]);
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

// ------------------------------------------------------------ 16-byte rows
// D a multiple of 8 and rows on 16-byte boundaries. A group of TPR threads owns a row, thread t
// the chunks of 8 columns t, t + TPR, ...; gamma and beta stay in registers. Both kernels are
// bound by HBM: each thread copies (cp.async) the chunks of its next RING - 1 rows into its own
// slots of a shared-memory ring, so the bytes in flight cost no registers, and a slot is
// refilled one row after it was read. Four neighbouring lanes hold a checkpoint block.
__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int ELEM, int TPR, int NV, bool RES>
struct FwdShape {
  static constexpr int THREADS = TPR < 256 ? 256 : TPR;
  static constexpr int W = ELEM == LNFP8_FP32 ? 2 : 1;           // 16-byte words per chunk
  static constexpr int WORDS = NV * W * (RES ? 2 : 1);           // per thread and row
  static constexpr int RING = WORDS <= 4 ? 4 : 3;
  static constexpr size_t SMEM = (size_t)RING * WORDS * THREADS * 16;
};

template <int ELEM, int TPR, int NV, bool CK, bool RES>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
ln_fwd_vec_kernel(const LnFwdParams p) {
  using S = FwdShape<ELEM, TPR, NV, RES>;
  constexpr int T = S::THREADS, GPB = T / TPR, W = S::W, RING = S::RING, P = RING - 1;
  __shared__ float2 xch[2 * T / 32];
  extern __shared__ uint4 ring[];  // [RING][WORDS][T]
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t stride = (int64_t)gridDim.x * GPB;
  constexpr int ES = ElemSize<ELEM>::value;
  auto issue = [&](int64_t r, int slot) {
    if (r < p.M) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + TPR * j) * 8;
        if (c < p.D) {
#pragma unroll
          for (int k = 0; k < W; ++k) {
            cp16(&ring[(slot * S::WORDS + j * W + k) * T + threadIdx.x], static_cast<const uint8_t*>(p.x) + (r * p.ldx + c) * ES + 16 * k);
            if constexpr (RES)
              cp16(&ring[(slot * S::WORDS + (NV + j) * W + k) * T + threadIdx.x],
                   static_cast<const uint8_t*>(p.resid) + (r * p.ldr + c) * ES + 16 * k);
          }
        }
      }
    }
    cp_commit();
  };
  int64_t row = (int64_t)blockIdx.x * GPB + g;
#pragma unroll
  for (int k = 0; k < P; ++k) issue(row + k * stride, k);
  float ga[NV][8], be[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + TPR * j) * 8;
    if (c < p.D) {
      load8_rt(p.gamma, p.param_elem, c, ga[j]);
      load8_rt(p.beta, p.param_elem, c, be[j]);
    }
  }
  const float inv_d = 1.0f / (float)p.D;
  int turn = 0, slot = 0;
  for (; row - g < p.M; row += stride) {  // the same trip count for every group of the block
    issue(row + P * stride, slot == 0 ? RING - 1 : slot - 1);
    cp_wait<P>();
    const bool active = row < p.M;
    float v[NV][8];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + TPR * j) * 8;
      const bool ok = active && c < p.D;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = 0.f;
      if (ok) {
        uint4 u[W];
#pragma unroll
        for (int k = 0; k < W; ++k) u[k] = ring[(slot * S::WORDS + j * W + k) * T + threadIdx.x];
        unpack8<ELEM>(u, v[j]);
        if constexpr (RES) {
          float r[8];
#pragma unroll
          for (int k = 0; k < W; ++k) u[k] = ring[(slot * S::WORDS + (NV + j) * W + k) * T + threadIdx.x];
          unpack8<ELEM>(u, r);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[j][k] += r[k];
          pack8<ELEM>(v[j], u);
          unpack8<ELEM>(u, v[j]);  // normalised as it is kept
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.xsum) + (row * p.D + c) * ES);
#pragma unroll
          for (int k = 0; k < W; ++k) dst[k] = u[k];
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[j][k];
    }
    slot = slot + 1 == RING ? 0 : slot + 1;
    const float mu = row_sum2<TPR>(s, 0.f, xch, turn).x * inv_d;
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if ((t + TPR * j) * 8 < p.D) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[j][k] -= mu;
          q = fmaf(v[j][k], v[j][k], q);
        }
      }
    const float rs = 1.0f / sqrtf(row_sum2<TPR>(q, 0.f, xch, turn).x * inv_d + p.eps);
    if (!active) continue;  // uniform over the row group
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + TPR * j) * 8;
      const bool in = c < p.D;
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] *= rs;
      if (in) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = fmaf(v[j][k], ga[j][k], be[j][k]);
        store8<ELEM>(p.y, row * p.ldy + c, y);
      }
      if constexpr (CK) {
        const uint32_t b = ckpt_byte(block_amax8(v[j]), p.dt);  // columns past D hold zeros
        if (in) {
          *reinterpret_cast<uint2*>(p.codes + row * p.D + c) = encode8(v[j], ckpt_inv_scale(b), p.dt);
          if ((t & 3) == 0) p.scales[row * p.pitch + (c >> 5)] = (uint8_t)b;
        }
      }
    }
    if (t == 0) {
      p.mu[row] = mu;
      p.rs[row] = rs;
    }
  }
  cp_wait<0>();
}

template <int ELEM, int TPR, int NV, bool CK, bool RES>
struct BwdShape {
  static constexpr int THREADS = TPR < 256 ? 256 : TPR;
  static constexpr int W = ELEM == LNFP8_FP32 ? 2 : 1;
  // 16-byte words per thread and row: dy, dres, x or the codes (8 bytes a chunk), then one word of
  // scalars (mu, rs) and the scale words
  static constexpr int X_WORDS = CK ? (NV + 1) / 2 : NV * W;
  static constexpr int WORDS = NV * W * (RES ? 2 : 1) + X_WORDS + 1;
  static constexpr int RING = WORDS <= 6 ? 4 : 3 * WORDS * THREADS * 16 <= 224 * 1024 ? 3 : 2;
  static constexpr size_t SMEM = (size_t)RING * WORDS * THREADS * 16;
  static_assert(SMEM <= 224 * 1024, "shared memory budget");
};

template <int ELEM, int TPR, int NV, bool CK, bool RES>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR < 512 ? 2 : 1)
ln_bwd_vec_kernel(const LnBwdParams p) {
  using S = BwdShape<ELEM, TPR, NV, CK, RES>;
  constexpr int T = S::THREADS, GPB = T / TPR, W = S::W, RING = S::RING, P = RING - 1;
  constexpr int X0 = NV * W, R0 = X0 + S::X_WORDS, S0 = S::WORDS - 1;  // word offsets in a slot: dy, x, dres, scalars
  static_assert(NV <= 2, "two scale words beside mu and rsigma");
  __shared__ float2 xch[2 * T / 32];
  extern __shared__ uint4 ring[];
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t stride = (int64_t)gridDim.x * GPB;
  constexpr int ES = ElemSize<ELEM>::value;
  auto at = [&](int slot, int w) { return &ring[(slot * S::WORDS + w) * T + threadIdx.x]; };
  auto issue = [&](int64_t r, int slot) {
    if (r < p.M) {
      uint32_t* sc = reinterpret_cast<uint32_t*>(at(slot, S0));
      cp4(sc, p.rs + r);
      if constexpr (!CK) cp4(sc + 1, p.mu + r);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + TPR * j) * 8;
        if (c < p.D) {
#pragma unroll
          for (int k = 0; k < W; ++k) {
            cp16(at(slot, j * W + k), static_cast<const uint8_t*>(p.dy) + (r * p.lddy + c) * ES + 16 * k);
            if constexpr (!CK) cp16(at(slot, X0 + j * W + k), static_cast<const uint8_t*>(p.x) + (r * p.ldx + c) * ES + 16 * k);
            if constexpr (RES) cp16(at(slot, R0 + j * W + k), static_cast<const uint8_t*>(p.dres) + (r * p.lddres + c) * ES + 16 * k);
          }
          if constexpr (CK) {
            cp8(reinterpret_cast<uint2*>(at(slot, X0)) + j, p.codes + r * p.D + c);
            cp4(sc + 2 + j, p.scales + r * p.pitch + ((c >> 7) << 2));
          }
        }
      }
    }
    cp_commit();
  };
  int64_t row = (int64_t)blockIdx.x * GPB + g;
#pragma unroll
  for (int k = 0; k < P; ++k) issue(row + k * stride, k);
  float ga[NV][8], accg[NV][8], accb[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int k = 0; k < 8; ++k) ga[j][k] = accg[j][k] = accb[j][k] = 0.f;
    const int c = (t + TPR * j) * 8;
    if (c < p.D) load8_rt(p.gamma, p.param_elem, c, ga[j]);
  }
  const float inv_d = 1.0f / (float)p.D;
  int turn = 0, slot = 0;
  for (; row - g < p.M; row += stride) {
    issue(row + P * stride, slot == 0 ? RING - 1 : slot - 1);
    cp_wait<P>();
    const bool active = row < p.M;
    float xh[NV][8], gg[NV][8];
    float rs = 0.f, s1 = 0.f, s2 = 0.f;
    if (active) rs = __uint_as_float(at(slot, S0)->x);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + TPR * j) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) xh[j][k] = gg[j][k] = 0.f;
      if (active && c < p.D) {
        uint4 u[W];
        float d[8];
#pragma unroll
        for (int k = 0; k < W; ++k) u[k] = *at(slot, j * W + k);
        unpack8<ELEM>(u, d);
        if constexpr (CK) {
          const uint4 sc = *at(slot, S0);
          decode8(reinterpret_cast<const uint2*>(at(slot, X0))[j], ckpt_scale(((j ? sc.w : sc.z) >> (((c >> 5) & 3) * 8)) & 0xFFu), p.dt, xh[j]);
        } else {
          const float mu = __uint_as_float(at(slot, S0)->y);
#pragma unroll
          for (int k = 0; k < W; ++k) u[k] = *at(slot, X0 + j * W + k);
          unpack8<ELEM>(u, xh[j]);
#pragma unroll
          for (int k = 0; k < 8; ++k) xh[j][k] = (xh[j][k] - mu) * rs;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          gg[j][k] = d[k] * ga[j][k];
          accg[j][k] = fmaf(d[k], xh[j][k], accg[j][k]);
          accb[j][k] += d[k];
          s1 += gg[j][k];
          s2 = fmaf(gg[j][k], xh[j][k], s2);
        }
      }
    }
    const float2 sums = row_sum2<TPR>(s1, s2, xch, turn);
    const float mg = sums.x * inv_d, nmx = -sums.y * inv_d;
    if (active) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + TPR * j) * 8;
        if (c >= p.D) continue;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = fmaf(nmx, xh[j][k], gg[j][k] - mg) * rs;
        if constexpr (RES) {
          uint4 u[W];
          float r[8];
#pragma unroll
          for (int k = 0; k < W; ++k) u[k] = *at(slot, R0 + j * W + k);
          unpack8<ELEM>(u, r);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] += r[k];
        }
        store8<ELEM>(p.dx, row * p.lddx + c, o);
      }
    }
    slot = slot + 1 == RING ? 0 : slot + 1;
  }
  cp_wait<0>();
  // column partials: the row groups add theirs in turn in the ring's memory
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
  float* red = reinterpret_cast<float*>(ring);
#pragma unroll 1
  for (int turn_g = 0; turn_g < GPB; ++turn_g) {
    if constexpr (GPB > 1) __syncthreads();
    if (g != turn_g) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + TPR * j) * 8;
      if (c >= p.D) continue;
#pragma unroll
      for (int h = 0; h < 4; ++h) {  // dgamma then dbeta, 4 columns at a time
        float* acc = h < 2 ? accg[j] + 4 * h : accb[j] + 4 * (h - 2);
        const int at_c = (h < 2 ? 0 : p.D) + c + 4 * (h & 1);
        float4 v = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (turn_g > 0) {
          const float4 o = *reinterpret_cast<const float4*>(red + at_c);
          v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        if (turn_g == GPB - 1) *reinterpret_cast<float4*>(part + at_c) = v;
        else *reinterpret_cast<float4*>(red + at_c) = v;
      }
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

template <int ELEM, bool CK>
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

template <int ELEM, bool CK>
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

bool al(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Resident blocks per SM, looked up once per kernel (the devices of a process are alike).
template <typename K>
int blocks_per_sm(K kernel, int threads, size_t smem) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
  return n;
}

template <int ELEM, bool CK, bool RES>
lnfp8_status fwd_vec(const LnFwdParams& p, cudaStream_t st) {
  auto go = [&](auto kernel, auto shape, int tpr) {
    using S = decltype(shape);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM) != cudaSuccess)
      return check_launch("layernorm_fwd: shared memory");
    const int gpb = S::THREADS / tpr;
    const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * blocks_per_sm(kernel, S::THREADS, S::SMEM));
    if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(S::THREADS), S::SMEM, st, p) != cudaSuccess) return check_launch("layernorm_fwd launch");
    return check_launch("layernorm_fwd");
  };
#define FWD(TPR, NV) go(ln_fwd_vec_kernel<ELEM, TPR, NV, CK, RES>, FwdShape<ELEM, TPR, NV, RES>(), TPR)
  if (p.D <= 256) return FWD(32, 1);
  if (p.D <= 512) return FWD(32, 2);
  if (p.D <= 1024) return FWD(64, 2);
  if (p.D <= 2048) return FWD(128, 2);
  if (p.D <= 4096) return FWD(256, 2);
  return FWD(512, 2);
#undef FWD
}

template <int ELEM, bool CK, bool RES>
lnfp8_status bwd_vec(const LnBwdParams& p, int* blocks_out, cudaStream_t st) {
  auto go = [&](auto kernel, auto shape, int tpr) {
    using S = decltype(shape);
    const int gpb = S::THREADS / tpr;
    const size_t smem = gpb > 1 ? std::max<size_t>(S::SMEM, 2 * (size_t)p.D * sizeof(float)) : S::SMEM;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return check_launch("layernorm_bwd: shared memory");
    const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * std::min(kBwdBlocksPerSm, blocks_per_sm(kernel, S::THREADS, smem)));
    *blocks_out = (int)blocks;
    if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(S::THREADS), smem, st, p) != cudaSuccess) return check_launch("layernorm_bwd launch");
    return check_launch("layernorm_bwd");
  };
#define BWD(TPR, NV) go(ln_bwd_vec_kernel<ELEM, TPR, NV, CK, RES>, BwdShape<ELEM, TPR, NV, CK, RES>(), TPR)
  if (p.D <= 256) return BWD(32, 1);
  if (p.D <= 512) return BWD(32, 2);
  if (p.D <= 1024) return BWD(64, 2);
  if (p.D <= 2048) return BWD(128, 2);
  if (p.D <= 4096) return BWD(256, 2);
  return BWD(512, 2);
#undef BWD
}

// Rows of 16-byte words up to 8192 columns take the vector kernels (beyond, and for any other
// width or alignment, the kernels above).
bool row_aligned(const void* p, int64_t ld, int es) { return al(p, 16) && ld * es % 16 == 0; }
template <int ELEM, bool CK>
lnfp8_status fwd(const LnFwdParams& p, cudaStream_t st) {
  constexpr int es = ElemSize<ELEM>::value;
  const bool vec = p.D % 8 == 0 && p.D <= 8192 && row_aligned(p.x, p.ldx, es) && row_aligned(p.y, p.ldy, es) && al(p.gamma, 16) && al(p.beta, 16) &&
                   (!p.resid || (row_aligned(p.resid, p.ldr, es) && al(p.xsum, 16))) && (!CK || al(p.codes, 8));
  if (!vec) return fwd_any<ELEM, CK>(p, st);
  return p.resid ? fwd_vec<ELEM, CK, true>(p, st) : fwd_vec<ELEM, CK, false>(p, st);
}
template <int ELEM, bool CK>
lnfp8_status bwd(const LnBwdParams& p, int* blocks_out, cudaStream_t st) {
  constexpr int es = ElemSize<ELEM>::value;
  const bool vec = p.D % 8 == 0 && p.D <= 8192 && row_aligned(p.dy, p.lddy, es) && row_aligned(p.dx, p.lddx, es) && al(p.gamma, 16) &&
                   (!p.dres || row_aligned(p.dres, p.lddres, es)) && (!CK ? row_aligned(p.x, p.ldx, es) : al(p.codes, 8));
  if (!vec) return bwd_any<ELEM, CK>(p, blocks_out, st);
  return p.dres ? bwd_vec<ELEM, CK, true>(p, blocks_out, st) : bwd_vec<ELEM, CK, false>(p, blocks_out, st);
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

#define BY_CKPT(ELEM, FN, ...) (a->ckpt.codes ? FN<ELEM, true>(__VA_ARGS__) : FN<ELEM, false>(__VA_ARGS__))
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
  p.dt = a->ckpt.dtype;
  LaunchScope ls("layernorm_fwd", st);
  return BY_ELEM(fwd, p, st);
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
  p.dt = a->ckpt.dtype;
  int blocks = 0;
  lnfp8_status s;
  {
    LaunchScope ls("layernorm_bwd", st);
    s = BY_ELEM(bwd, p, &blocks, st);
  }
  if (s != LNFP8_OK) return s;
  return colsum_launch(p.part, blocks, 2 * p.D, p.D, a->dgamma, a->dbeta, st);
}

}  // namespace lnfp8
