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
#include "cp_async.cuh"
#include "internal.h"
#include "kernel_setup.cuh"
#include "rowmath.cuh"

#include <algorithm>

namespace lnfp8 {
namespace {

constexpr int kMaxD = 16384;

// Sums of two values over W neighbouring lanes (a warp: in 6 shuffles): the halves first swap, so that each
// goes on with one of the two.
template <int W = 32>
__device__ __forceinline__ float2 warp_sum2(float a, float b) {
  const bool hi = (threadIdx.x & (W / 2)) != 0;
  float v = (hi ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, hi ? a : b, W / 2);
#pragma unroll
  for (int o = W / 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const float w = __shfl_xor_sync(0xFFFFFFFFu, v, W / 2);
  return hi ? make_float2(w, v) : make_float2(v, w);
}

// Sum over the TPR threads of a row group; every thread gets the result. `xch`
// holds two buffers of 32 floats per group, used in turn (`turn` counts the sums),
// so that one barrier per sum is enough.
template <int TPR>
__device__ __forceinline__ void group_sync() {
  if constexpr (TPR == 1024) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"((int)threadIdx.x / TPR + 1), "r"(TPR) : "memory");
}
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* xch, int& turn) {
  const float2 s = warp_sum2<TPR < 32 ? TPR : 32>(a, b);
  if constexpr (TPR <= 32) {
    return s;
  } else {
    constexpr int W = TPR / 32;
    const int group = threadIdx.x / TPR, w = (threadIdx.x % TPR) / 32, lane = threadIdx.x & 31;
    float2* buf = xch + (group * 2 + (turn++ & 1)) * W;
    if (lane == 0) buf[w] = s;
    group_sync<TPR>();
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
      return warp_sum2(v.x, v.y);
    }
  }
}
template <int TPR>
__device__ __forceinline__ float row_sum(float a, float2* xch, int& turn) {
  if constexpr (TPR < 32) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    return a;
  }
  a = warp_sum(a);
  if constexpr (TPR <= 32) {
    return a;
  } else {
    constexpr int W = TPR / 32;
    const int group = threadIdx.x / TPR, w = (threadIdx.x % TPR) / 32, lane = threadIdx.x & 31;
    float* buf = reinterpret_cast<float*>(xch + (group * 2 + (turn++ & 1)) * W);
    if (lane == 0) buf[w] = a;
    group_sync<TPR>();
    if constexpr (W <= 8) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) s += buf[i];
      return s;
    } else {
      return warp_sum(lane < W ? buf[lane] : 0.f);
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
  int64_t step, xstep, rstep, ystep, hstep, cstep, sstep;  // rows a group moves on by; the same in bytes of each tensor
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
  int64_t step, dstep, xstep, rstep, ostep, cstep, sstep;
};

// ------------------------------------------------------------ any width, any alignment
// A group of TPR threads owns a row; thread t holds columns t, t + TPR, ... (so that a warp reads 32
// neighbours and a checkpoint block is one warp's value i). Addresses are one pointer per tensor
// and row, the columns compile-time offsets. A column or row that a thread does not have is replaced by one that
// exists, and its value by zero, so that no load waits for a condition. Bound by a row's latency: nothing is copied
// ahead. 8191 x 1001 fp16: forward 12 us, backward 46 -> 20. HOLD: gamma and beta stay in registers.
template <int ELEM, int TPR, int NE, bool CK>  // CK: with a checkpoint
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
ln_fwd_any_kernel(const LnFwdParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, ES = ElemSize<ELEM>::value;
  constexpr int GPB = kThreads / TPR;
  constexpr bool HOLD = NE <= 8;
  __shared__ float2 xch[2 * kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const float inv_d = 1.0f / (float)p.D;
  const int n = (p.D - t + TPR - 1) / TPR;  // this thread's columns (0 or fewer: none)
  const int tc = min(t, p.D - 1);           // a column to load in place of those it has not
  float ga[HOLD ? NE : 1], be[HOLD ? NE : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) {
        ga[i] = load_elem_rt(p.gamma, p.param_elem, t + TPR * i);
        be[i] = load_elem_rt(p.beta, p.param_elem, t + TPR * i);
      }
  }
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * GPB; row0 < p.M; row0 += (int64_t)gridDim.x * GPB) {
    const int64_t row = row0 + g;
    const bool active = row < p.M;
    float v[NE];
    float s = 0.f;
    const int64_t rowc = active ? row : p.M - 1;
    const uint8_t* xr = static_cast<const uint8_t*>(p.x) + (rowc * p.ldx + tc) * ES;
    uint32_t xb[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) xb[i] = load_bits<ELEM>(xr, i < n ? TPR * i : 0);
    if (!p.resid) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = active && i < n ? bits_value<ELEM>(xb[i]) : 0.f;
    } else {
      const uint8_t* rr = static_cast<const uint8_t*>(p.resid) + (rowc * p.ldr + tc) * ES;
      uint32_t rb[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) rb[i] = load_bits<ELEM>(rr, i < n ? TPR * i : 0);
      uint8_t* hr = static_cast<uint8_t*>(p.xsum) + (row * p.D + t) * ES;
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = active && i < n ? round_elem<ELEM>(bits_value<ELEM>(xb[i]) + bits_value<ELEM>(rb[i])) : 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (active && i < n) store_elem<ELEM>(hr, TPR * i, v[i]);
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) s += v[i];
    const float mu = row_sum<TPR>(s, xch, turn) * inv_d;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) {
        v[i] -= mu;
        q = fmaf(v[i], v[i], q);
      }
    const float rs = rsqrt_nr(row_sum<TPR>(q, xch, turn) * inv_d + p.eps);
    if (!active) continue;  // uniform over the row group; the barriers above are behind it
    uint8_t* yr = static_cast<uint8_t*>(p.y) + (row * p.ldy + t) * ES;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      v[i] *= rs;  // columns past D hold zeros
      if (i < n) {
        const float gi = HOLD ? ga[HOLD ? i : 0] : load_elem_rt(p.gamma, p.param_elem, t + TPR * i);
        const float bi = HOLD ? be[HOLD ? i : 0] : load_elem_rt(p.beta, p.param_elem, t + TPR * i);
        store_elem<ELEM>(yr, TPR * i, fmaf(v[i], gi, bi));
      }
    }
    if constexpr (CK) {
      uint8_t *cr = p.codes + row * p.D + t, *sr = p.scales + row * p.pitch + (t >> 5);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const uint32_t b = ckpt_byte(__reduce_max_sync(0xFFFFFFFFu, abs_bits(v[i])), p.dt);
        const uint32_t code = fp8x2(v[i] * ckpt_inv_scale(b), 0.f, p.dt);
        if (i < n) {
          cr[TPR * i] = (uint8_t)code;
          if ((t & 31) == 0) sr[TPR / 32 * i] = (uint8_t)b;
        }
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
  constexpr int kThreads = TPR < 256 ? 256 : TPR, ES = ElemSize<ELEM>::value;
  constexpr int GPB = kThreads / TPR;
  __shared__ float2 xch[2 * kThreads / 32];
  // [2][D]: where several row groups add their column sums, or, with more than 8 columns a thread, where the
  // sums are kept from the start (in registers 2048 x 16384 spilled and took 318 us)
  extern __shared__ float colred[];
  constexpr bool SACC = NE > 8;
  pdl_wait();
  pdl_launch_dependents();
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const float inv_d = 1.0f / (float)p.D;
  const int n = (p.D - t + TPR - 1) / TPR, tc = min(t, p.D - 1);
  constexpr bool HOLD = NE <= 8;  // gamma in registers
  float accg[SACC ? 1 : NE], accb[SACC ? 1 : NE], ga[HOLD ? NE : 1];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if constexpr (SACC) {
      if (i < n) colred[t + TPR * i] = colred[p.D + t + TPR * i] = 0.f;
    } else {
      accg[i] = accb[i] = 0.f;
    }
    if constexpr (HOLD)
      if (i < n) ga[i] = load_elem_rt(p.gamma, p.param_elem, t + TPR * i);
  }
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * GPB; row0 < p.M; row0 += (int64_t)gridDim.x * GPB) {
    const int64_t row = row0 + g;
    const bool active = row < p.M;
    const int64_t rowc = active ? row : p.M - 1;
    const float rs = p.rs[rowc];
    const float mu = CK ? 0.f : p.mu[rowc];
    float xh[NE], gg[NE];
    float s1 = 0.f, s2 = 0.f;
    const uint8_t* dr = static_cast<const uint8_t*>(p.dy) + (rowc * p.lddy + tc) * ES;
    const uint8_t* xr = CK ? p.codes + rowc * p.D + tc : static_cast<const uint8_t*>(p.x) + (rowc * p.ldx + tc) * ES;
    const uint8_t* sr = p.scales + rowc * p.pitch + (tc >> 5);
    uint32_t db[NE], xb[NE], sb[CK ? NE : 1], rb[SACC ? 1 : NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {  // every load of the row first
      const int at = i < n ? TPR * i : 0;
      db[i] = load_bits<ELEM>(dr, at);
      if constexpr (CK) {
        xb[i] = xr[at];
        sb[i] = sr[at / 32];
      } else {
        xb[i] = load_bits<ELEM>(xr, at);
      }
    }
    const uint8_t* rr = static_cast<const uint8_t*>(p.dres) + (rowc * p.lddres + tc) * ES;
    if constexpr (!SACC) {
      if (p.dres) {
#pragma unroll
        for (int i = 0; i < NE; ++i) rb[i] = load_bits<ELEM>(rr, i < n ? TPR * i : 0);
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const bool in = active && i < n;
      const float x = CK ? fp8x2_to_f32(xb[i], p.dt).x * ckpt_scale(sb[CK ? i : 0]) : (bits_value<ELEM>(xb[i]) - mu) * rs;
      const float d = in ? bits_value<ELEM>(db[i]) : 0.f;
      xh[i] = in ? x : 0.f;
      if constexpr (SACC) {
        if (in) {
          colred[t + TPR * i] = fmaf(d, xh[i], colred[t + TPR * i]);
          colred[p.D + t + TPR * i] += d;
        }
      } else {
        accg[i] = fmaf(d, xh[i], accg[i]);
        accb[i] += d;
      }
      gg[i] = in ? d * (HOLD ? ga[HOLD ? i : 0] : load_elem_rt(p.gamma, p.param_elem, tc + (i < n ? TPR * i : 0))) : 0.f;
      s1 += gg[i];
      s2 = fmaf(gg[i], xh[i], s2);
    }
    const float2 sums = row_sum2<TPR>(s1, s2, xch, turn);
    if (!active) continue;  // uniform over the row group
    const float mg = sums.x * inv_d, mgx = sums.y * inv_d;
    uint8_t* orow = static_cast<uint8_t*>(p.dx) + (row * p.lddx + t) * ES;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      if (i >= n) continue;
      const float o = fmaf(-mgx, xh[i], gg[i] - mg) * rs;
      if constexpr (SACC) store_elem<ELEM>(orow, TPR * i, p.dres ? o + load_elem<ELEM>(rr, TPR * i) : o);
      else store_elem<ELEM>(orow, TPR * i, p.dres ? o + bits_value<ELEM>(rb[i]) : o);
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
      part[c] = SACC ? colred[c] : accg[SACC ? 0 : i];
      part[p.D + c] = SACC ? colred[p.D + c] : accb[SACC ? 0 : i];
    }
  }
}

// ------------------------------------------------------------ 16-byte rows
// D a multiple of 8 and rows on 16-byte boundaries. A group of TPR threads owns a row. Both kernels are
// bound by HBM: each thread copies (cp.async) the words of its next RING - 1 rows into its own
// slots of a shared-memory ring, so the bytes in flight cost no registers, and a slot is
// refilled one row after it was read. Neighbouring lanes hold a checkpoint block. 16 columns a thread
// measured best (8 or 32, or 96 threads for 768 columns, up to 2x slower backward: fewer columns share a
// row's reductions, more cost occupancy); up to 256 columns 8 or 16 lanes hold a row, and a warp several
// (262144 x 128: forward 55 -> 24 us, backward 111 -> 38). bf16, 16384 x 2048, with residual and checkpoint: forward
// 52 us, 5.8 TB/s, 85% of a copy; backward 44 us with its column sums, 80%.
// A thread's NV 16-byte words of a row are words t, t + TPR, ... (EPC columns each: 8 of a 16-bit type, 4 of
// fp32), so that every access of a warp is of whole sectors. HOLD: gamma and beta stay in registers; beyond
// 16 columns a thread they are read again for each row.
template <int ELEM>
struct Word {
  static constexpr int EPC = ELEM == LNFP8_FP32 ? 4 : 8;
  static constexpr int LANES = 32 / EPC;  // that hold a checkpoint block
};

template <int ELEM, int TPR, int NV, bool RES>
struct FwdShape {
  static constexpr int THREADS = TPR < 256 ? 256 : TPR;
  static constexpr int WORDS = NV * (RES ? 2 : 1);  // per thread and row
  static constexpr int RING = WORDS <= 4 ? 4 : 3 * WORDS * THREADS * 16 <= 224 * 1024 ? 3 : 2;
  static constexpr size_t SMEM = (size_t)RING * WORDS * THREADS * 16;
};

template <int ELEM, int TPR, int NV, bool CK, bool RES>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR < 512 ? 3 : 1)
ln_fwd_vec_kernel(const LnFwdParams p) {
  using S = FwdShape<ELEM, TPR, NV, RES>;
  constexpr int T = S::THREADS, GPB = T / TPR, RING = S::RING, P = RING - 1;
  constexpr int EPC = Word<ELEM>::EPC, PP = EPC / 2, ES = ElemSize<ELEM>::value;
  constexpr bool HOLD = NV * EPC <= 16;
  __shared__ float2 xch[2 * T / 32];
  extern __shared__ uint4 ring[];  // [RING][WORDS][T]
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  pdl_wait();
  pdl_launch_dependents();
  constexpr uint32_t WB = T * 16, SB = S::WORDS * WB;  // bytes of a word of all threads, of a slot
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
  int64_t row = (int64_t)blockIdx.x * GPB + g;
  // this thread's first word in the row to be loaded next: the pointers run ahead of `row`
  const uint8_t* xp = static_cast<const uint8_t*>(p.x) + row * p.ldx * ES + t * 16;
  const uint8_t* rp = RES ? static_cast<const uint8_t*>(p.resid) + row * p.ldr * ES + t * 16 : nullptr;
  auto issue = [&](int64_t r, uint32_t slot) {
    if (r < p.M) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if ((t + TPR * j) * EPC < p.D) {
          cp16(slot + j * WB, xp + TPR * j * 16);
          if constexpr (RES) cp16(slot + (NV + j) * WB, rp + TPR * j * 16);
        }
      }
      xp += p.xstep;
      if constexpr (RES) rp += p.rstep;
    }
    cp_commit();
  };
#pragma unroll
  for (int k = 0; k < P; ++k) issue(row + k * p.step, mine + k * SB);
  uint64_t ga[HOLD ? NV : 1][PP], be[HOLD ? NV : 1][PP];  // pairs of columns
  if constexpr (HOLD) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + TPR * j) * EPC;
      if (c < p.D) {
        load_params<EPC>(p.gamma, p.param_elem, c, ga[j]);
        load_params<EPC>(p.beta, p.param_elem, c, be[j]);
      }
    }
  }
  const float inv_d = 1.0f / (float)p.D;
  int turn = 0;
  uint32_t slot = mine, last = mine + P * SB;  // the row's slot; the one read before it, filled next
  // the word's place in the outputs, advanced row by row
  uint8_t* yp = static_cast<uint8_t*>(p.y) + row * p.ldy * ES + t * 16;
  uint8_t* hp = RES ? static_cast<uint8_t*>(p.xsum) + row * p.D * ES + t * 16 : nullptr;
  uint8_t* cp = CK ? p.codes + row * p.D + t * EPC : nullptr;
  uint8_t* sp8 = CK ? p.scales + row * p.pitch + t / Word<ELEM>::LANES : nullptr;
  for (; row - g < p.M; row += p.step) {  // the same trip count for every group of the block
    issue(row + P * p.step, last);
    cp_wait<P>();
    const bool active = row < p.M;
    uint64_t v[NV][PP];
    uint64_t s2 = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < PP; ++k) v[j][k] = 0;
      if (active && (t + TPR * j) * EPC < p.D) {
        unpack_word<ELEM>(lds16(slot + j * WB), v[j]);
        if constexpr (RES) {
          uint64_t r[PP];
          unpack_word<ELEM>(lds16(slot + (NV + j) * WB), r);
#pragma unroll
          for (int k = 0; k < PP; ++k) v[j][k] = add_2(v[j][k], r[k]);
          const uint4 u = pack_word<ELEM>(v[j]);
          unpack_word<ELEM>(u, v[j]);  // normalised as it is kept
          *reinterpret_cast<uint4*>(hp + TPR * j * 16) = u;
        }
      }
#pragma unroll
      for (int k = 0; k < PP; ++k) s2 = add_2(s2, v[j][k]);
    }
    last = slot;
    slot = slot == mine + P * SB ? mine : slot + SB;
    const float2 sp = upk(s2);
    const float mu = row_sum<TPR>(sp.x + sp.y, xch, turn) * inv_d;
    const uint64_t mu2 = pk(mu, mu);
    uint64_t q2 = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if ((t + TPR * j) * EPC < p.D) {
#pragma unroll
        for (int k = 0; k < PP; ++k) {
          v[j][k] = sub_2(v[j][k], mu2);
          q2 = fma_2(v[j][k], v[j][k], q2);
        }
      }
    const float2 qp = upk(q2);
    const float rs = rsqrt_nr(row_sum<TPR>(qp.x + qp.y, xch, turn) * inv_d + p.eps);
    if (TPR >= 32 && !active) continue;  // uniform over the row group; narrower groups meet in the shuffles below
    const uint64_t rs2 = pk(rs, rs);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + TPR * j) * EPC;
      const bool in = c < p.D && (TPR >= 32 || active);
#pragma unroll
      for (int k = 0; k < PP; ++k) v[j][k] = mul_2(v[j][k], rs2);
      if (in) {
        uint64_t y[PP];
        if constexpr (!HOLD) {
          load_params<EPC>(p.gamma, p.param_elem, c, ga[0]);
          load_params<EPC>(p.beta, p.param_elem, c, be[0]);
        }
#pragma unroll
        for (int k = 0; k < PP; ++k) y[k] = fma_2(v[j][k], ga[HOLD ? j : 0][k], be[HOLD ? j : 0][k]);
        *reinterpret_cast<uint4*>(yp + TPR * j * 16) = pack_word<ELEM>(y);
      }
      if constexpr (CK) {  // columns past D hold zeros
        const uint32_t b = ckpt_byte(EPC == 8 ? block_amax8(v[j]) : block_amax4(v[j]), p.dt);
        if (in) {
          encode_pairs<EPC>(v[j], ckpt_inv_scale(b), p.dt, cp + TPR * j * EPC);
          if (t % Word<ELEM>::LANES == 0) sp8[TPR / Word<ELEM>::LANES * j] = (uint8_t)b;
        }
      }
    }
    if (t == 0 && (TPR >= 32 || active)) {
      p.mu[row] = mu;
      p.rs[row] = rs;
    }
    yp += p.ystep;
    if constexpr (RES) hp += p.hstep;
    if constexpr (CK) {
      cp += p.cstep;
      sp8 += p.sstep;
    }
  }
  cp_wait<0>();
}

template <int ELEM, int TPR, int NV, bool CK, bool RES>
struct BwdShape {
  static constexpr int THREADS = TPR < 256 ? 256 : TPR;
  // bytes per thread and row, each kind an array over the threads (so that a warp's accesses fill whole
  // lines of banks): dy, x or the codes, dres, then rsigma and mu or the scale words
  static constexpr int X_OFF = NV * 16, R_OFF = X_OFF + (CK ? NV * Word<ELEM>::EPC : NV * 16);
  static constexpr int S_OFF = R_OFF + (RES ? NV * 16 : 0), BYTES = S_OFF + 4 + (CK ? NV * 4 : 4);
  static constexpr int RING = 4 * BYTES * THREADS <= 104 * 1024 ? 4 : 3 * BYTES * THREADS <= 224 * 1024 ? 3 : 2;
  static constexpr size_t SMEM = (size_t)RING * BYTES * THREADS;
  static_assert(SMEM <= 224 * 1024, "shared memory budget");
};

template <int ELEM, int TPR, int NV, bool CK, bool RES>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR < 512 ? 2 : 1)
ln_bwd_vec_kernel(const LnBwdParams p) {
  using S = BwdShape<ELEM, TPR, NV, CK, RES>;
  constexpr int T = S::THREADS, GPB = T / TPR, RING = S::RING, P = RING - 1;
  constexpr int EPC = Word<ELEM>::EPC, PP = EPC / 2, ES = ElemSize<ELEM>::value, LANES = Word<ELEM>::LANES;
  __shared__ float2 xch[2 * T / 32];
  extern __shared__ uint4 ring[];  // [RING][BYTES * T]
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  pdl_wait();
  pdl_launch_dependents();
  constexpr uint32_t SB = S::BYTES * T;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t t16 = threadIdx.x * 16, tq = S::X_OFF * T + threadIdx.x * EPC, t4 = S::S_OFF * T + threadIdx.x * 4;
  int64_t row = (int64_t)blockIdx.x * GPB + g;
  // this thread's first word in the row to be loaded next: the pointers run ahead of `row`
  const uint8_t* dp = static_cast<const uint8_t*>(p.dy) + row * p.lddy * ES + t * 16;
  const uint8_t* xp = CK ? p.codes + row * p.D + t * EPC : static_cast<const uint8_t*>(p.x) + row * p.ldx * ES + t * 16;
  // the scale byte of word j is byte t / LANES + TPR / LANES j of the row: in the word at bp + scale_word(j), from bit
  // byte + scale_byte(j) on
  constexpr bool kWide = TPR % (4 * LANES) == 0;  // else TPR is 1 or 2 blocks
  auto scale_word = [](int j) { return kWide ? TPR / LANES * j : TPR / LANES * j / 4 * 4; };
  auto scale_byte = [](int j) { return kWide ? 0 : TPR / LANES * j % 4 * 8; };
  const uint8_t* bp = CK ? p.scales + row * p.pitch + t / (4 * LANES) * 4 : nullptr;
  const uint8_t* rp = RES ? static_cast<const uint8_t*>(p.dres) + row * p.lddres * ES + t * 16 : nullptr;
  const float* mp = p.mu + row;
  const float* sp = p.rs + row;
  static_assert(kWide || 4 * LANES % TPR == 0, "a group's blocks do not cross a scale word");
  auto issue = [&](int64_t r, uint32_t slot) {
    if (r < p.M) {
      cp4(slot + t4, sp);
      if constexpr (!CK) cp4(slot + t4 + 4 * T, mp);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if ((t + TPR * j) * EPC < p.D) {
          cp16(slot + t16 + j * 16 * T, dp + TPR * j * 16);
          if constexpr (!CK) cp16(slot + t16 + (S::X_OFF + j * 16) * T, xp + TPR * j * 16);
          if constexpr (RES) cp16(slot + t16 + (S::R_OFF + j * 16) * T, rp + TPR * j * 16);
          if constexpr (CK) {
            if constexpr (EPC == 8) cp8(slot + tq + j * 8 * T, xp + TPR * j * 8);
            else cp4(slot + tq + j * 4 * T, xp + TPR * j * 4);
            cp4(slot + t4 + (4 + 4 * j) * T, bp + scale_word(j));
          }
        }
      }
      dp += p.dstep;
      xp += CK ? p.cstep : p.xstep;
      if constexpr (CK) bp += p.sstep;
      if constexpr (RES) rp += p.rstep;
      if constexpr (!CK) mp += p.step;
      sp += p.step;
    }
    cp_commit();
  };
  // words past D, and the slots of a group that gets no row at all, are read but never filled
#pragma unroll
  for (int k = 0; k < RING; ++k) {
    sts4(base + k * SB + t4, 0u);
    sts4(base + k * SB + t4 + 4 * T, 0u);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if ((t + TPR * j) * EPC < p.D && row < p.M) continue;
      sts16_zero(base + k * SB + t16 + j * 16 * T);
      if constexpr (!CK) sts16_zero(base + k * SB + t16 + (S::X_OFF + j * 16) * T);
      if constexpr (CK) {
#pragma unroll
        for (int q = 0; q < EPC; q += 4) sts4(base + k * SB + tq + j * EPC * T + q, 0u);
        sts4(base + k * SB + t4 + (4 + 4 * j) * T, 0u);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < P; ++k) issue(row + k * p.step, base + k * SB);
  uint64_t ga[NV][PP], accg[NV][PP], accb[NV][PP];  // pairs of columns
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int k = 0; k < PP; ++k) ga[j][k] = accg[j][k] = accb[j][k] = 0;
    const int c = (t + TPR * j) * EPC;
    if (c < p.D) load_params<EPC>(p.gamma, p.param_elem, c, ga[j]);
  }
  const float inv_d = 1.0f / (float)p.D;
  int turn = 0;
  uint32_t slot = base, last = base + P * SB;
  const int byte = t / LANES % 4 * 8;  // of this thread's scale in each of its words
  uint8_t* op = static_cast<uint8_t*>(p.dx) + row * p.lddx * ES + t * 16;
  for (; row - g < p.M; row += p.step) {
    issue(row + P * p.step, last);
    cp_wait<P>();
    const bool active = row < p.M;
    uint64_t xh[NV][PP], gg[NV][PP];
    uint64_t a1 = 0, a2 = 0;
    // every word of the row first; those past D hold zeros from the start, and a group without a row
    // goes through the motions on an old one
    uint4 du[NV], xu[NV];
    uint32_t sw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      du[j] = lds16(slot + t16 + j * 16 * T);
      if constexpr (!CK) xu[j] = lds16(slot + t16 + (S::X_OFF + j * 16) * T);
      if constexpr (CK) {
        if constexpr (EPC == 8) {
          const uint2 q = lds8(slot + tq + j * 8 * T);
          xu[j].x = q.x;
          xu[j].y = q.y;
        } else {
          xu[j].x = lds4(slot + tq + j * 4 * T);
        }
        sw[j] = lds4(slot + t4 + (4 + 4 * j) * T);
      }
    }
    const float rs = __uint_as_float(lds4(slot + t4));
    const float mu = CK ? 0.f : __uint_as_float(lds4(slot + t4 + 4 * T));
    const uint64_t rs2 = pk(rs, rs), mu2 = pk(mu, mu);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t d[PP];
      unpack_word<ELEM>(du[j], d);
      if constexpr (CK) {
        const float s = ckpt_scale((sw[j] >> (byte + scale_byte(j))) & 0xFFu);
        if constexpr (EPC == 8) {
          decode8(make_uint2(xu[j].x, xu[j].y), s, p.dt, xh[j]);
        } else {
          const float2 a = fp8x2_to_f32(xu[j].x & 0xFFFFu, p.dt), b = fp8x2_to_f32(xu[j].x >> 16, p.dt);
          xh[j][0] = mul_2(pk(a.x, a.y), pk(s, s));
          xh[j][1] = mul_2(pk(b.x, b.y), pk(s, s));
        }
      } else {
        unpack_word<ELEM>(xu[j], xh[j]);
#pragma unroll
        for (int k = 0; k < PP; ++k) xh[j][k] = mul_2(sub_2(xh[j][k], mu2), rs2);
      }
#pragma unroll
      for (int k = 0; k < PP; ++k) {
        gg[j][k] = mul_2(d[k], ga[j][k]);
        a1 = add_2(a1, gg[j][k]);
        a2 = fma_2(gg[j][k], xh[j][k], a2);
      }
      if (active) {
#pragma unroll
        for (int k = 0; k < PP; ++k) {
          accg[j][k] = fma_2(d[k], xh[j][k], accg[j][k]);
          accb[j][k] = add_2(accb[j][k], d[k]);
        }
      }
    }
    const float2 p1 = upk(a1), p2 = upk(a2);
    const float2 sums = row_sum2<TPR>(p1.x + p1.y, p2.x + p2.y, xch, turn);
    const float mg = sums.x * inv_d, nmx = -sums.y * inv_d;
    if (active) {
      const uint64_t mg2 = pk(mg, mg), nmx2 = pk(nmx, nmx);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if ((t + TPR * j) * EPC >= p.D) continue;
        uint64_t o[PP];
#pragma unroll
        for (int k = 0; k < PP; ++k) o[k] = mul_2(fma_2(nmx2, xh[j][k], sub_2(gg[j][k], mg2)), rs2);
        if constexpr (RES) {
          uint64_t r[PP];
          unpack_word<ELEM>(lds16(slot + t16 + (S::R_OFF + j * 16) * T), r);
#pragma unroll
          for (int k = 0; k < PP; ++k) o[k] = add_2(o[k], r[k]);
        }
        *reinterpret_cast<uint4*>(op + TPR * j * 16) = pack_word<ELEM>(o);
      }
    }
    op += p.ostep;
    last = slot;
    slot = slot == base + P * SB ? base : slot + SB;
  }
  cp_wait<0>();
  // column partials: the row groups of a warp by shuffles, then the others in turn in the ring's memory
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
  float* red = reinterpret_cast<float*>(ring);
  constexpr int TURNS = TPR < 32 ? T / 32 : GPB;
  if constexpr (TPR < 32) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < PP; ++k)
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1) {
          accg[j][k] = add_2(accg[j][k], __shfl_xor_sync(0xFFFFFFFFu, accg[j][k], o));
          accb[j][k] = add_2(accb[j][k], __shfl_xor_sync(0xFFFFFFFFu, accb[j][k], o));
        }
  }
#pragma unroll 1
  for (int turn_g = 0; turn_g < TURNS; ++turn_g) {
    if constexpr (TURNS > 1) __syncthreads();
    if (TPR < 32 ? (int)threadIdx.x >> 5 != turn_g || (threadIdx.x & 31) >= TPR : g != turn_g) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + TPR * j) * EPC;
      if (c >= p.D) continue;
#pragma unroll
      for (int h = 0; h < EPC / 2; ++h) {  // dgamma then dbeta, 4 columns at a time
        const int q = h % (EPC / 4);
        const uint64_t* acc = h < EPC / 4 ? accg[j] + 2 * q : accb[j] + 2 * q;
        const int at_c = (h < EPC / 4 ? 0 : p.D) + c + 4 * q;
        const float2 lo = upk(acc[0]), hi = upk(acc[1]);
        float4 v = make_float4(lo.x, lo.y, hi.x, hi.y);
        if (turn_g > 0) {
          const float4 o = *reinterpret_cast<const float4*>(red + at_c);
          v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        if (turn_g == TURNS - 1) *reinterpret_cast<float4*>(part + at_c) = v;
        else *reinterpret_cast<float4*>(red + at_c) = v;
      }
    }
  }
}

// Sums over n partial rows of `cols` floats in a fixed order: 32 columns per block, warp w adds rows
// w, w + 32, ..., then the warps' sums are added over the lanes of a warp. A few hundred rows leave
// each thread about ten loads, all in flight at once: 304 x 1536, cold, took 9.9 us with 8 warps a
// block, 8.6 with 32.
__global__ void __launch_bounds__(1024) colsum_kernel(const float* __restrict__ part, int n, int cols, int split,
                                                      float* __restrict__ a, float* __restrict__ b) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 10
    for (int i = w; i < n; i += 32) s += __ldcs(part + (int64_t)i * cols + c);
  }
  red[w][lane] = s;
  __syncthreads();
  s = warp_sum(red[lane][w]);  // warp w: column w of the block
  const int cw = blockIdx.x * 32 + w;
  if (lane == 0 && cw < cols) {
    if (cw < split) a[cw] = s;
    else b[cw - split] = s;
  }
}

// The most blocks an SM gets of the backward's row pass, each of which leaves a partial row of column sums: two
// (measured best for the vector kernels), or three of up to 2048 columns, where the kernels of any width are bound by
// the latency of a row (41654 x 457 bf16 52 us with two, 39 with three).
int bwd_blocks_per_sm(int64_t D) { return D <= 2048 ? 3 : 2; }
constexpr int kBwdVecBlocksPerSm = 2;

template <int ELEM, bool CK>
lnfp8_status fwd_any(const LnFwdParams& p, cudaStream_t st) {
  auto go = [&](auto kernel, int tpr) {
    const int threads = tpr < 256 ? 256 : tpr, gpb = threads / tpr;
    const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * (2048 / threads));
    if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, p) != cudaSuccess) return check_launch("layernorm_fwd launch");
    return check_launch("layernorm_fwd");
  };
  if (p.D <= 256) return go(ln_fwd_any_kernel<ELEM, 32, 8, CK>, 32);
  if (p.D <= 512) return go(ln_fwd_any_kernel<ELEM, 64, 8, CK>, 64);
  if (p.D <= 1024) return go(ln_fwd_any_kernel<ELEM, 128, 8, CK>, 128);
  if (p.D <= 2048) return go(ln_fwd_any_kernel<ELEM, 256, 8, CK>, 256);
  if (p.D <= 4096) return go(ln_fwd_any_kernel<ELEM, 512, 8, CK>, 512);
  if (p.D <= 8192) return go(ln_fwd_any_kernel<ELEM, 1024, 8, CK>, 1024);
  return go(ln_fwd_any_kernel<ELEM, 1024, 16, CK>, 1024);
}

template <int ELEM, int TPR, int NE, bool CK>
lnfp8_status bwd_any_launch(const LnBwdParams& p, int* blocks_out, cudaStream_t st) {
  constexpr auto kernel = ln_bwd_any_kernel<ELEM, TPR, NE, CK>;
  constexpr int threads = TPR < 256 ? 256 : TPR, gpb = threads / TPR;
  constexpr bool sums = gpb > 1 || NE > 8;  // in shared memory
  int bps = 1;
  const lnfp8_status s = kernel_setup<kernel>(threads, sums ? 2 * TPR * NE * sizeof(float) : 0, &bps, "layernorm_bwd: kernel set-up");
  if (s != LNFP8_OK) return s;
  const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * std::min(bwd_blocks_per_sm(p.D), bps));
  *blocks_out = (int)blocks;
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), sums ? 2 * (size_t)p.D * sizeof(float) : 0, st, p) != cudaSuccess)
    return check_launch("layernorm_bwd launch");
  return check_launch("layernorm_bwd");
}

template <int ELEM, bool CK>
lnfp8_status bwd_any(const LnBwdParams& p, int* blocks_out, cudaStream_t st) {
  if (p.D <= 256) return bwd_any_launch<ELEM, 32, 8, CK>(p, blocks_out, st);
  if (p.D <= 512) return bwd_any_launch<ELEM, 64, 8, CK>(p, blocks_out, st);
  if (p.D <= 1024) return bwd_any_launch<ELEM, 128, 8, CK>(p, blocks_out, st);
  if (p.D <= 2048) return bwd_any_launch<ELEM, 256, 8, CK>(p, blocks_out, st);
  if (p.D <= 4096) return bwd_any_launch<ELEM, 512, 8, CK>(p, blocks_out, st);
  if (p.D <= 8192) return bwd_any_launch<ELEM, 1024, 8, CK>(p, blocks_out, st);
  return bwd_any_launch<ELEM, 1024, 16, CK>(p, blocks_out, st);
}

bool al(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <int ELEM, int TPR, int NV, bool CK, bool RES>
lnfp8_status fwd_vec_launch(const LnFwdParams& p, cudaStream_t st) {
  using S = FwdShape<ELEM, TPR, NV, RES>;
  constexpr auto kernel = ln_fwd_vec_kernel<ELEM, TPR, NV, CK, RES>;
  int bps = 1;
  const lnfp8_status s = kernel_setup<kernel>(S::THREADS, S::SMEM, &bps, "layernorm_fwd: kernel set-up");
  if (s != LNFP8_OK) return s;
  constexpr int gpb = S::THREADS / TPR, es = ElemSize<ELEM>::value;
  const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * bps);
  LnFwdParams q = p;
  q.step = blocks * gpb;
  q.xstep = q.step * p.ldx * es;
  q.rstep = q.step * p.ldr * es;
  q.ystep = q.step * p.ldy * es;
  q.hstep = q.step * p.D * es;
  q.cstep = q.step * p.D;
  q.sstep = q.step * p.pitch;
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(S::THREADS), S::SMEM, st, q) != cudaSuccess) return check_launch("layernorm_fwd launch");
  return check_launch("layernorm_fwd");
}

// 16 columns a thread; the forward's last step takes 32.
template <int ELEM, bool CK, bool RES>
lnfp8_status fwd_vec(const LnFwdParams& p, cudaStream_t st) {
  constexpr int NV = 16 / Word<ELEM>::EPC;
  if (p.D <= 128) return fwd_vec_launch<ELEM, 8, NV, CK, RES>(p, st);
  if (p.D <= 256) return fwd_vec_launch<ELEM, 16, NV, CK, RES>(p, st);
  if (p.D <= 512) return fwd_vec_launch<ELEM, 32, NV, CK, RES>(p, st);
  if (p.D <= 1024) return fwd_vec_launch<ELEM, 64, NV, CK, RES>(p, st);
  if (p.D <= 2048) return fwd_vec_launch<ELEM, 128, NV, CK, RES>(p, st);
  if (p.D <= 4096) return fwd_vec_launch<ELEM, 256, NV, CK, RES>(p, st);
  if constexpr (ELEM == LNFP8_FP32 && RES) return fwd_vec_launch<ELEM, 512, NV, CK, RES>(p, st);
  else return p.D <= 8192 ? fwd_vec_launch<ELEM, 512, NV, CK, RES>(p, st) : fwd_vec_launch<ELEM, 512, 2 * NV, CK, RES>(p, st);
}

template <int ELEM, int TPR, int NV, bool CK, bool RES>
lnfp8_status bwd_vec_launch(const LnBwdParams& p, int* blocks_out, cudaStream_t st) {
  using S = BwdShape<ELEM, TPR, NV, CK, RES>;
  static_assert(S::SMEM >= TPR * NV * Word<ELEM>::EPC * 2 * sizeof(float), "the column partials reuse the ring");
  constexpr auto kernel = ln_bwd_vec_kernel<ELEM, TPR, NV, CK, RES>;
  int bps = 1;
  const lnfp8_status s = kernel_setup<kernel>(S::THREADS, S::SMEM, &bps, "layernorm_bwd: kernel set-up");
  if (s != LNFP8_OK) return s;
  constexpr int gpb = S::THREADS / TPR, es = ElemSize<ELEM>::value;
  const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * std::min(kBwdVecBlocksPerSm, bps));
  *blocks_out = (int)blocks;
  LnBwdParams q = p;
  q.step = blocks * gpb;
  q.dstep = q.step * p.lddy * es;
  q.xstep = q.step * p.ldx * es;
  q.rstep = q.step * p.lddres * es;
  q.ostep = q.step * p.lddx * es;
  q.cstep = q.step * p.D;
  q.sstep = q.step * p.pitch;
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(S::THREADS), S::SMEM, st, q) != cudaSuccess) return check_launch("layernorm_bwd launch");
  return check_launch("layernorm_bwd");
}

template <int ELEM, bool CK, bool RES>
lnfp8_status bwd_vec(const LnBwdParams& p, int* blocks_out, cudaStream_t st) {
  constexpr int NV = 16 / Word<ELEM>::EPC;
  if (p.D <= 128) return bwd_vec_launch<ELEM, 8, NV, CK, RES>(p, blocks_out, st);
  if (p.D <= 256) return bwd_vec_launch<ELEM, 16, NV, CK, RES>(p, blocks_out, st);
  if (p.D <= 512) return bwd_vec_launch<ELEM, 32, NV, CK, RES>(p, blocks_out, st);
  if (p.D <= 1024) return bwd_vec_launch<ELEM, 64, NV, CK, RES>(p, blocks_out, st);
  if (p.D <= 2048) return bwd_vec_launch<ELEM, 128, NV, CK, RES>(p, blocks_out, st);
  if (p.D <= 4096) return bwd_vec_launch<ELEM, 256, NV, CK, RES>(p, blocks_out, st);
  return bwd_vec_launch<ELEM, 512, NV, CK, RES>(p, blocks_out, st);
}

// Rows of 16-byte words take the vector kernels up to 16384 columns forward (8192 in fp32 with a residual, whose
// ring would not fit) and 8192 backward; all others the kernels above.
bool row_aligned(const void* p, int64_t ld, int es) { return al(p, 16) && ld * es % 16 == 0; }
template <int ELEM, bool CK>
lnfp8_status fwd(const LnFwdParams& p, cudaStream_t st) {
  constexpr int es = ElemSize<ELEM>::value;
  const bool vec = p.D % 8 == 0 && (p.D <= 8192 || !(ELEM == LNFP8_FP32 && p.resid)) && row_aligned(p.x, p.ldx, es) && row_aligned(p.y, p.ldy, es) && al(p.gamma, 16) && al(p.beta, 16) &&
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
  return min64(M, (int64_t)num_sms() * bwd_blocks_per_sm(D)) * 2 * D * (int64_t)sizeof(float);
}

lnfp8_status colsum_launch(const float* part, int n, int cols, int split, float* a, float* b, cudaStream_t st) {
  LaunchScope ls("colsum", st);
  if (launch_pdl(colsum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, st, part, n, cols, split, a, b) != cudaSuccess)
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
