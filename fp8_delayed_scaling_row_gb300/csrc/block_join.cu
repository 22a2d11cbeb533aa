// The join of a block's output with the residual stream, from one block to the next (a transformer layer around the
// modules of the TE tutorial, code block 2: dropout and residual add behind each sub-layer, a norm in front of the next):
//   forward   n = norm1(x) g1 + b1, h = T(r + s drop(gate n)), y = T(norm2(h) g2 + b2)
//   backward  dH = dh + rs2 (q - [mean(q)] - hhat mean(q hhat)), q = dy g2; dt = s drop'(dH), dn = gate dt,
//             dx = T(rs1 (u - [mean(u)] - xhat mean(u xhat))), u = dn g1; dr = T(dH)
//             ([mean]: layer norms only)
// Each part is optional. All arithmetic is fp32. The forward folds s, gate, 1 / (1 - p), g1 and b1 into one factor and one
// summand a column: t = xhat a + c where kept. Of column sums the backward needs four at most, since
// dgate = sum dt n = g1 A + b1 B, dg1 = gate A, db1 = gate B with A = sum dt xhat, B = sum dt.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kernel_setup.cuh"
#include "philox.cuh"
#include "rowmath.cuh"
#include "rowsum.cuh"

namespace lnfp8 {
namespace {

struct JoinFwdParams {
  const void* x;
  const void* resid;
  const void* g1;
  const void* b1;
  const void* gate;
  const void* g2;
  const void* b2;
  void* h;
  void* y;
  float* mu1;
  float* rs1;
  float* mu2;
  float* rs2;
  int64_t M, ldx, ldr, ldh, ldy;
  int D, param_elem, layer;
  float eps, scale;  // scale: s / (1 - p)
  DropParams drop;
};

struct JoinBwdParams {
  const void* dh;
  const void* dy;
  const void* x;
  const void* h;
  const void* g1;
  const void* gate;
  const void* g2;
  const float* mu1;
  const float* rs1;
  const float* mu2;
  const float* rs2;
  void* dx;
  void* dres;
  float* part;  // [blocks][4][D]: sums of dy hhat, dy, dt xhat, dt, as far as `sums` has their bits
  int64_t M, lddh, lddy, ldx, ldh, lddx, lddres;
  int D, param_elem, layer, sums;
  float scale;
  DropParams drop;
};

// A column's parameter, or `none` where there is no such vector.
__device__ __forceinline__ float param_or(const void* p, int elem, int c, float none) { return p ? load_elem_rt(p, elem, c) : none; }

// ------------------------------------------------------------ any width, any alignment
// A group of TPR threads owns a row; thread t holds columns t, t + TPR, ..., so that a warp's value i is 32 neighbours:
// four groups of draws. Lane q draws for group q of the warp's NE * 4, and the draws pass through shared memory. A column
// or row that a thread does not have is replaced by one that exists, and its value by zero.
template <int NE>
__device__ __forceinline__ void any_draws(uint16_t* bits, const DropKey& key, int t, int tpr, uint32_t row) {
  const int lane = threadIdx.x & 31, w0 = t & ~31;
  __syncwarp();  // the last row's draws have been read
#pragma unroll
  for (int k = 0; k < NE / 8; ++k) {
    const int q = lane + 32 * k;
    *reinterpret_cast<uint4*>(bits + 8 * q) = drop_bits(key, (uint32_t)(w0 + tpr * (q >> 2)) / 8 + (q & 3), row);
  }
  __syncwarp();
}

template <int ELEM, int TPR, int NE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) join_fwd_any_kernel(const JoinFwdParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, ES = ElemSize<ELEM>::value, GPB = kThreads / TPR;
  __shared__ float2 xch[2 * kThreads / 32];
  __shared__ __align__(16) uint16_t draws[kThreads / 32][32 * NE];
  pdl_wait();
  pdl_launch_dependents();
  drop_save(p.drop);
  const DropKey key = drop_key(p.drop);
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR, lane = threadIdx.x & 31;
  uint16_t* bits = draws[threadIdx.x >> 5];
  const float inv_d = 1.0f / (float)p.D;
  const int n = (p.D - t + TPR - 1) / TPR;  // this thread's columns (0 or fewer: none)
  const int tc = min(t, p.D - 1);           // a column to load in place of those it has not
  int turn = 0;
  // mean and reciprocal deviation of a row; v becomes the normalised values
  auto normalise = [&](float* v, float& mu, float& rs) {
    mu = 0.f;
    if (p.layer) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) s += v[i];
      mu = row_sum<TPR>(s, xch, turn) * inv_d;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) {
        v[i] -= mu;
        q = fmaf(v[i], v[i], q);
      }
    rs = rsqrt_nr(row_sum<TPR>(q, xch, turn) * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] *= rs;
  };
  for (int64_t row0 = (int64_t)blockIdx.x * GPB; row0 < p.M; row0 += (int64_t)gridDim.x * GPB) {
    const int64_t row = row0 + g;
    const bool active = row < p.M;
    const int64_t rowc = active ? row : p.M - 1;
    const uint8_t* xr = static_cast<const uint8_t*>(p.x) + (rowc * p.ldx + tc) * ES;
    const uint8_t* rr = static_cast<const uint8_t*>(p.resid) + (rowc * p.ldr + tc) * ES;
    uint32_t xb[NE], rb[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) xb[i] = load_bits<ELEM>(xr, i < n ? TPR * i : 0);
#pragma unroll
    for (int i = 0; i < NE; ++i) rb[i] = 0u;
    if (p.resid) {
#pragma unroll
      for (int i = 0; i < NE; ++i) rb[i] = load_bits<ELEM>(rr, i < n ? TPR * i : 0);
    }
    float v[NE], mu, rs;
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] = active && i < n ? bits_value<ELEM>(xb[i]) : 0.f;
    if (p.g1) {
      normalise(v, mu, rs);
      if (t == 0 && active) {
        p.rs1[row] = rs;
        if (p.layer) p.mu1[row] = mu;
      }
    }
    if (p.drop.cut) any_draws<NE>(bits, key, t, TPR, (uint32_t)row);
    uint8_t* hr = static_cast<uint8_t*>(p.h) + (row * p.ldh + t) * ES;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = tc + (i < n ? TPR * i : 0);
      const float f = p.scale * param_or(p.gate, p.param_elem, c, 1.f);
      const float tv = fmaf(v[i], f * param_or(p.g1, p.param_elem, c, 1.f), f * param_or(p.b1, p.param_elem, c, 0.f));
      const bool keep = p.drop.cut == 0 || bits[32 * i + lane] >= p.drop.cut;
      const float sum = bits_value<ELEM>(rb[i]) + (keep ? tv : 0.f);
      v[i] = active && i < n ? round_elem<ELEM>(sum) : 0.f;
      if (active && i < n) store_elem<ELEM>(hr, TPR * i, v[i]);
    }
    if (!p.g2) continue;
    normalise(v, mu, rs);
    if (!active) continue;  // uniform over the row group; the barriers above are behind it
    if (t == 0) {
      p.rs2[row] = rs;
      if (p.layer) p.mu2[row] = mu;
    }
    uint8_t* yr = static_cast<uint8_t*>(p.y) + (row * p.ldy + t) * ES;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      if (i >= n) continue;
      const int c = t + TPR * i;
      store_elem<ELEM>(yr, TPR * i, fmaf(v[i], load_elem_rt(p.g2, p.param_elem, c), param_or(p.b2, p.param_elem, c, 0.f)));
    }
  }
}

template <int ELEM, int TPR, int NE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) join_bwd_any_kernel(const JoinBwdParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, ES = ElemSize<ELEM>::value, GPB = kThreads / TPR;
  __shared__ float2 xch[2 * kThreads / 32];
  __shared__ __align__(16) uint16_t draws[kThreads / 32][32 * NE];
  extern __shared__ float colred[];  // [D]: where several row groups add their column sums
  pdl_wait();
  pdl_launch_dependents();
  const DropKey key = drop_key(p.drop);
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR, lane = threadIdx.x & 31;
  uint16_t* bits = draws[threadIdx.x >> 5];
  const float inv_d = 1.0f / (float)p.D;
  const int n = (p.D - t + TPR - 1) / TPR, tc = min(t, p.D - 1);
  float acc[4][NE];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[k][i] = 0.f;
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * GPB; row0 < p.M; row0 += (int64_t)gridDim.x * GPB) {
    const int64_t row = row0 + g;
    const bool active = row < p.M;
    const int64_t rowc = active ? row : p.M - 1;
    auto load = [&](const void* src, int64_t ld, float* v) {
      const uint8_t* r = static_cast<const uint8_t*>(src) + (rowc * ld + tc) * ES;
      uint32_t b[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) b[i] = load_bits<ELEM>(r, i < n ? TPR * i : 0);
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = active && i < n ? bits_value<ELEM>(b[i]) : 0.f;
    };
    float d[NE], xh[NE];  // the gradient on its way down; normalised values
#pragma unroll
    for (int i = 0; i < NE; ++i) d[i] = 0.f;
    if (p.dh) load(p.dh, p.lddh, d);
    if (p.g2) {
      float q[NE];
      load(p.dy, p.lddy, q);
      load(p.h, p.ldh, xh);
      const float rs = p.rs2[rowc], mu = p.layer ? p.mu2[rowc] : 0.f;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        xh[i] = active && i < n ? (xh[i] - mu) * rs : 0.f;
        acc[0][i] = fmaf(q[i], xh[i], acc[0][i]);
        acc[1][i] += q[i];
        q[i] *= load_elem_rt(p.g2, p.param_elem, tc + (i < n ? TPR * i : 0));
        s1 += q[i];
        s2 = fmaf(q[i], xh[i], s2);
      }
      const float2 s = row_sum2<TPR>(s1, s2, xch, turn);
      const float mq = p.layer ? s.x * inv_d : 0.f, mqx = s.y * inv_d;
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] += fmaf(-mqx, xh[i], q[i] - mq) * rs;
    }
    if (p.dres && active) {
      uint8_t* o = static_cast<uint8_t*>(p.dres) + (row * p.lddres + t) * ES;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (i < n) store_elem<ELEM>(o, TPR * i, d[i]);
    }
    if (p.drop.cut) any_draws<NE>(bits, key, t, TPR, (uint32_t)row);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const bool keep = p.drop.cut == 0 || bits[32 * i + lane] >= p.drop.cut;
      d[i] = keep && active && i < n ? d[i] * p.scale : 0.f;  // dt
    }
    float rs = 1.f;
    if (p.g1 || p.gate) {
      load(p.x, p.ldx, xh);
      if (p.g1) {
        rs = p.rs1[rowc];
        const float mu = p.layer ? p.mu1[rowc] : 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) xh[i] = active && i < n ? (xh[i] - mu) * rs : 0.f;
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        acc[2][i] = fmaf(d[i], xh[i], acc[2][i]);
        acc[3][i] += d[i];
      }
    }
    float mu_ = 0.f, mux = 0.f;
    if (p.g1 || p.gate) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = tc + (i < n ? TPR * i : 0);
        d[i] *= param_or(p.gate, p.param_elem, c, 1.f) * param_or(p.g1, p.param_elem, c, 1.f);
      }
    }
    if (p.g1) {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        s1 += d[i];
        s2 = fmaf(d[i], xh[i], s2);
      }
      const float2 s = row_sum2<TPR>(s1, s2, xch, turn);
      mu_ = p.layer ? s.x * inv_d : 0.f;
      mux = s.y * inv_d;
    }
    if (!active) continue;  // uniform over the row group
    uint8_t* o = static_cast<uint8_t*>(p.dx) + (row * p.lddx + t) * ES;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) store_elem<ELEM>(o, TPR * i, p.g1 ? fmaf(-mux, xh[i], d[i] - mu_) * rs : d[i]);
  }
  // this block's column partials: the row groups add theirs in turn
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!(p.sums >> k & 1)) continue;
    float* part = p.part + ((int64_t)blockIdx.x * 4 + k) * p.D;
#pragma unroll 1
    for (int turn_g = 0; turn_g < GPB; ++turn_g) {
      if constexpr (GPB > 1) __syncthreads();
      if (g != turn_g) continue;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = t + TPR * i;
        if (c >= p.D) continue;
        const float v = turn_g ? colred[c] + acc[k][i] : acc[k][i];
        if (turn_g == GPB - 1) part[c] = v;
        else colred[c] = v;
      }
    }
  }
}

// The column sums of n partial rows in a fixed order (32 columns a block, warp w adds rows w, w + 32, ..., then the warps'
// sums are added over the lanes), and what the gradients make of them.
struct JoinSumParams {
  const float* part;
  const void* g1;
  const void* b1;
  const void* gate;
  float* dg1;
  float* db1;
  float* dgate;
  float* dg2;
  float* db2;
  int n, D, param_elem, sums;
};
__global__ void __launch_bounds__(1024) join_sum_kernel(const JoinSumParams p) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, cw = blockIdx.x * 32 + w;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!(p.sums >> k & 1)) continue;
    if (c < p.D) {
#pragma unroll 10
      for (int i = w; i < p.n; i += 32) s[k] += __ldcs(p.part + ((int64_t)i * 4 + k) * p.D + c);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!(p.sums >> k & 1)) continue;
    __syncthreads();
    red[w][lane] = s[k];
    __syncthreads();
    s[k] = warp_sum(red[lane][w]);  // warp w: column w of the block
  }
  if (lane != 0 || cw >= p.D) return;
  if (p.dg2) p.dg2[cw] = s[0];
  if (p.db2) p.db2[cw] = s[1];
  const float f = param_or(p.gate, p.param_elem, cw, 1.f);
  if (p.dg1) p.dg1[cw] = f * s[2];
  if (p.db1) p.db1[cw] = f * s[3];
  if (p.dgate) p.dgate[cw] = p.g1 ? fmaf(load_elem_rt(p.g1, p.param_elem, cw), s[2], p.b1 ? load_elem_rt(p.b1, p.param_elem, cw) * s[3] : 0.f) : s[2];
}

// ------------------------------------------------------------ host side
template <int ELEM>
lnfp8_status fwd_any(const JoinFwdParams& p, cudaStream_t st) {
  auto go = [&](auto kernel, int tpr) {
    const int threads = tpr < 256 ? 256 : tpr, gpb = threads / tpr;
    const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * (2048 / threads));
    if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, p) != cudaSuccess) return check_launch("block_join_fwd launch");
    return check_launch("block_join_fwd");
  };
  if (p.D <= 256) return go(join_fwd_any_kernel<ELEM, 32, 8>, 32);
  if (p.D <= 512) return go(join_fwd_any_kernel<ELEM, 64, 8>, 64);
  if (p.D <= 1024) return go(join_fwd_any_kernel<ELEM, 128, 8>, 128);
  if (p.D <= 2048) return go(join_fwd_any_kernel<ELEM, 256, 8>, 256);
  if (p.D <= 4096) return go(join_fwd_any_kernel<ELEM, 512, 8>, 512);
  if (p.D <= 8192) return go(join_fwd_any_kernel<ELEM, 1024, 8>, 1024);
  return go(join_fwd_any_kernel<ELEM, 1024, 16>, 1024);
}

constexpr int kBwdBlocksPerSm = 2;  // at most: each leaves partial rows of the column sums

template <int ELEM, int TPR, int NE>
lnfp8_status bwd_any_launch(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  constexpr auto kernel = join_bwd_any_kernel<ELEM, TPR, NE>;
  constexpr int threads = TPR < 256 ? 256 : TPR, gpb = threads / TPR;
  constexpr size_t smem = gpb > 1 ? TPR * NE * sizeof(float) : 0;
  int bps = 1;
  const lnfp8_status s = kernel_setup<kernel>(threads, smem, &bps, "block_join_bwd: kernel set-up");
  if (s != LNFP8_OK) return s;
  const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * std::min(kBwdBlocksPerSm, bps));
  *blocks_out = (int)blocks;
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), smem, st, p) != cudaSuccess) return check_launch("block_join_bwd launch");
  return check_launch("block_join_bwd");
}
template <int ELEM>
lnfp8_status bwd_any(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  if (p.D <= 256) return bwd_any_launch<ELEM, 32, 8>(p, blocks_out, st);
  if (p.D <= 512) return bwd_any_launch<ELEM, 64, 8>(p, blocks_out, st);
  if (p.D <= 1024) return bwd_any_launch<ELEM, 128, 8>(p, blocks_out, st);
  if (p.D <= 2048) return bwd_any_launch<ELEM, 256, 8>(p, blocks_out, st);
  if (p.D <= 4096) return bwd_any_launch<ELEM, 512, 8>(p, blocks_out, st);
  if (p.D <= 8192) return bwd_any_launch<ELEM, 1024, 8>(p, blocks_out, st);
  return bwd_any_launch<ELEM, 1024, 16>(p, blocks_out, st);
}

}  // namespace

lnfp8_status block_join_fwd_launch(const lnfp8_block_join_fwd_args* a, cudaStream_t st) {
  if (a->M == 0) return LNFP8_OK;
  JoinFwdParams p = {};
  p.x = a->x;
  p.resid = a->residual;
  p.g1 = a->post_gamma;
  p.b1 = a->post_beta;
  p.gate = a->gate;
  p.g2 = a->pre_gamma;
  p.b2 = a->pre_beta;
  p.h = a->h;
  p.y = a->y;
  p.mu1 = a->post_mu;
  p.rs1 = a->post_rsigma;
  p.mu2 = a->pre_mu;
  p.rs2 = a->pre_rsigma;
  p.M = a->M;
  p.ldx = a->ldx;
  p.ldr = a->ld_residual;
  p.ldh = a->ldh;
  p.ldy = a->ldy;
  p.D = (int)a->D;
  p.param_elem = a->param_elem;
  p.layer = a->norm == LNFP8_NORM_LAYER;
  p.eps = a->eps;
  p.scale = (float)(a->scale * drop_scale(a->drop));
  p.drop = drop_params(a->drop);
  LaunchScope ls("block_join_fwd", st);
  if (a->elem == LNFP8_BF16) return fwd_any<LNFP8_BF16>(p, st);
  return a->elem == LNFP8_FP16 ? fwd_any<LNFP8_FP16>(p, st) : fwd_any<LNFP8_FP32>(p, st);
}

int64_t block_join_bwd_ws_bytes(int64_t M, int64_t D) {
  if (M == 0) return 0;
  return min64(M, (int64_t)num_sms() * kBwdBlocksPerSm) * 4 * D * (int64_t)sizeof(float);
}

lnfp8_status block_join_bwd_launch(const lnfp8_block_join_bwd_args* a, cudaStream_t st) {
  if (a->M == 0) {
    for (float* v : {a->dpost_gamma, a->dpost_beta, a->dgate, a->dpre_gamma, a->dpre_beta})
      if (v && cudaMemsetAsync(v, 0, a->D * sizeof(float), st) != cudaSuccess) return check_launch("block_join_bwd: clearing gradients");
    return LNFP8_OK;
  }
  JoinBwdParams p = {};
  p.dh = a->dh;
  p.dy = a->dy;
  p.x = a->x;
  p.h = a->h;
  p.g1 = a->post_gamma;
  p.gate = a->gate;
  p.g2 = a->pre_gamma;
  p.mu1 = a->post_mu;
  p.rs1 = a->post_rsigma;
  p.mu2 = a->pre_mu;
  p.rs2 = a->pre_rsigma;
  p.dx = a->dx;
  p.dres = a->dresidual;
  p.part = static_cast<float*>(a->workspace);
  p.M = a->M;
  p.lddh = a->ld_dh;
  p.lddy = a->ld_dy;
  p.ldx = a->ldx;
  p.ldh = a->ldh;
  p.lddx = a->ld_dx;
  p.lddres = a->ld_dresidual;
  p.D = (int)a->D;
  p.param_elem = a->param_elem;
  p.layer = a->norm == LNFP8_NORM_LAYER;
  p.scale = (float)(a->scale * drop_scale(a->drop));
  p.drop = drop_params(a->drop);
  p.sums = (a->dpre_gamma ? 1 : 0) | (a->dpre_beta ? 2 : 0) | (a->dpost_gamma || a->dgate ? 4 : 0) |
           (a->dpost_beta || (a->dgate && a->post_beta) ? 8 : 0);
  int blocks = 0;
  lnfp8_status s;
  {
    LaunchScope ls("block_join_bwd", st);
    s = a->elem == LNFP8_BF16   ? bwd_any<LNFP8_BF16>(p, &blocks, st)
        : a->elem == LNFP8_FP16 ? bwd_any<LNFP8_FP16>(p, &blocks, st)
                                : bwd_any<LNFP8_FP32>(p, &blocks, st);
  }
  if (s != LNFP8_OK || p.sums == 0) return s;
  JoinSumParams q;
  q.part = p.part;
  q.g1 = a->post_gamma;
  q.b1 = a->post_beta;
  q.gate = a->gate;
  q.dg1 = a->dpost_gamma;
  q.db1 = a->dpost_beta;
  q.dgate = a->dgate;
  q.dg2 = a->dpre_gamma;
  q.db2 = a->dpre_beta;
  q.n = blocks;
  q.D = p.D;
  q.param_elem = p.param_elem;
  q.sums = p.sums;
  LaunchScope ls("block_join_sum", st);
  if (launch_pdl(join_sum_kernel, dim3((unsigned)((p.D + 31) / 32)), dim3(1024), 0, st, q) != cudaSuccess)
    return check_launch("block_join_bwd launch");
  return check_launch("block_join_bwd: column sums");
}

}  // namespace lnfp8
