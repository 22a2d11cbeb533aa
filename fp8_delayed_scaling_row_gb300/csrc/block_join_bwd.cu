// The backward of the join of a block's output with the residual stream (block_join.cuh).
#include <algorithm>

#include "block_join.cuh"

namespace lnfp8 {
namespace {

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
  float* part;  // [blocks][4][D]: sums of dy hhat, dy, dt xhat / scale, dt / scale, as far as `sums` has their bits
  int64_t M, lddh, lddy, ldx, ldh, lddx, lddres;
  int D, param_elem, layer, sums;
  float scale;
  DropParams drop;
  int64_t step, dhstep, dystep, xstep, hstep, dxstep, drstep;
};

template <int ELEM, int TPR, int NE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR <= 256 ? 2 : 1) join_bwd_any_kernel(const JoinBwdParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, ES = ElemSize<ELEM>::value, GPB = kThreads / TPR;
  __shared__ float2 xch[2 * kThreads / 32];
  __shared__ __align__(16) uint16_t draws[kThreads / 32][32 * NE];
  // [D]: where several row groups add their column sums; or, from 1024 threads a row on, which have 64 registers each, [3][D] where
  // the first three of them are kept from the start (2048 x 16384 bf16 with two RMS norms 428 -> 401 us)
  extern __shared__ float colred[];
  constexpr bool SACC = TPR >= 1024;
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
    for (int i = 0; i < NE; ++i) {
      acc[k][i] = 0.f;
      if (SACC && k < 3 && i < n) colred[k * p.D + t + TPR * i] = 0.f;
    }
  auto add = [&](int k, int i, float v) {  // (zero where the thread has no column or no row)
    if (!SACC || k == 3) acc[k][i] += v;
    else if (i < n && (p.sums >> k & 1)) colred[k * p.D + t + TPR * i] += v;
  };
  constexpr bool HOLD = TPR <= 512;  // the columns' factors stay in registers
  float fg[HOLD ? NE : 1], fa[HOLD ? NE : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = tc + (i < n ? TPR * i : 0);
      fg[i] = param_or(p.g2, p.param_elem, c, 0.f);
      fa[i] = p.scale * param_or(p.gate, p.param_elem, c, 1.f) * param_or(p.g1, p.param_elem, c, 1.f);
    }
  }
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * GPB; row0 < p.M; row0 += (int64_t)gridDim.x * GPB) {
    const int64_t row = row0 + g;
    const bool active = row < p.M;
    const int64_t rowc = active ? row : p.M - 1;
    auto fetch = [&](const void* src, int64_t ld, uint32_t* b) {
      const uint8_t* r = static_cast<const uint8_t*>(src) + (rowc * ld + tc) * ES;
#pragma unroll
      for (int i = 0; i < NE; ++i) b[i] = load_bits<ELEM>(r, i < n ? TPR * i : 0);
    };
    auto value = [&](const uint32_t* b, float* v) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = active && i < n ? bits_value<ELEM>(b[i]) : 0.f;
    };
    // every load of the row first, where there are registers for them
    constexpr bool FIRST = TPR <= 512;
    uint32_t b0[NE], b1[NE], b2[FIRST ? NE : 1], b3[FIRST ? NE : 1];
    if (p.g2) {
      fetch(p.dy, p.lddy, b0);
      fetch(p.h, p.ldh, b1);
    }
    if constexpr (FIRST) {
      if (p.dh) fetch(p.dh, p.lddh, b2);
      if (p.g1 || p.gate) fetch(p.x, p.ldx, b3);
    }
    float d[NE], xh[NE];  // the gradient on its way down; normalised values
#pragma unroll
    for (int i = 0; i < NE; ++i) d[i] = 0.f;
    if (p.g2) {
      float q[NE];
      value(b0, q);
      value(b1, xh);
      const float rs = p.rs2[rowc], mu = p.layer ? p.mu2[rowc] : 0.f;
      float s1 = 0.f, s2 = 0.f, f[HOLD ? 1 : NE];
      if constexpr (!HOLD) load_params_any<TPR, NE>(p.g2, p.param_elem, tc, n, f);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        xh[i] = active && i < n ? (xh[i] - mu) * rs : 0.f;
        add(0, i, q[i] * xh[i]);
        add(1, i, q[i]);
        if constexpr (HOLD) q[i] *= fg[i];
        else q[i] *= f[i];
        s1 += q[i];
        s2 = fmaf(q[i], xh[i], s2);
      }
      const float2 s = row_sum2<TPR>(s1, s2, xch, turn);
      const float mq = p.layer ? s.x * inv_d : 0.f, mqx = s.y * inv_d;
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] = fmaf(-mqx, xh[i], q[i] - mq) * rs;
    }
    if (p.dh) {
      float r[NE];
      if constexpr (FIRST) {
        value(b2, r);
      } else {
        fetch(p.dh, p.lddh, b0);
        value(b0, r);
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] += r[i];
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
      d[i] = keep && active && i < n ? d[i] : 0.f;
    }
    float rs = 1.f;
    if (p.g1 || p.gate) {
      if constexpr (FIRST) {
        value(b3, xh);
      } else {
        fetch(p.x, p.ldx, b0);
        value(b0, xh);
      }
      if (p.g1) {
        rs = p.rs1[rowc];
        const float mu = p.layer ? p.mu1[rowc] : 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) xh[i] = active && i < n ? (xh[i] - mu) * rs : 0.f;
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        add(2, i, d[i] * xh[i]);
        add(3, i, d[i]);
      }
    }
    float mu_ = 0.f, mux = 0.f;
    if constexpr (HOLD) {
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] *= fa[i];
    } else {
      float f[NE];
      if (p.gate) {
        load_params_any<TPR, NE>(p.gate, p.param_elem, tc, n, f);
#pragma unroll
        for (int i = 0; i < NE; ++i) d[i] *= f[i];
      }
      if (p.g1) {
        load_params_any<TPR, NE>(p.g1, p.param_elem, tc, n, f);
#pragma unroll
        for (int i = 0; i < NE; ++i) d[i] *= f[i];
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] *= p.scale;
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
        const float v = SACC && k < 3 ? colred[k * p.D + c] : turn_g ? colred[c] + acc[k][i] : acc[k][i];
        if (turn_g == GPB - 1) part[c] = v;
        else colred[c] = v;
      }
    }
  }
}

template <int ELEM, int TPR, int NV, bool FULL, int T, bool SHIFT>
struct JoinBwdShape {
  // bytes per thread and row, each kind an array over the threads: dy, h, dh, x, then rs2, rs1 and, FULL, mu2, mu1
  // (SHIFT: a word more a row of each tensor)
  static constexpr int TENSOR = (T * NV + (SHIFT ? T / TPR : 0)) * 16, STATS = 4 * TENSOR;
  static constexpr int SLOT = STATS + (FULL ? 16 : 8) * T, FACTORS = 2 * TPR * NV * Word<ELEM>::EPC * 4;
  static constexpr int FIT = (kVecSmem - FACTORS) / SLOT, RING = FIT < 4 ? FIT : 4;
  static constexpr size_t SMEM = (size_t)RING * SLOT + FACTORS;
  static_assert(RING >= 2, "shared memory budget");
};

// FULL: with means, and with the sums of dy and dt (for the betas).
template <int ELEM, int TPR, int NV, bool FULL, int T, bool SHIFT>
__global__ void __launch_bounds__(T, 1) join_bwd_vec_kernel(const JoinBwdParams p) {
  using S = JoinBwdShape<ELEM, TPR, NV, FULL, T, SHIFT>;
  constexpr int GPB = T / TPR, RING = S::RING, P = RING - 1;
  constexpr int EPC = Word<ELEM>::EPC, PP = EPC / 2, ES = ElemSize<ELEM>::value;
  // with four sums of 32 columns the normalised values are made again from the row's words wherever they are used
  constexpr bool REMAKE = NV == 4;
  __shared__ float2 xch[2 * T / 32];
  extern __shared__ uint4 ring[];  // [RING][SLOT bytes], then the factors pre_gamma, scale gate post_gamma
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  pdl_wait();
  pdl_launch_dependents();
  constexpr uint32_t WB = SHIFT ? TPR * 16 : T * 16, TB = S::TENSOR, SB = S::SLOT;  // bytes to a thread's next word, of a tensor, of a slot
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t t16 = (SHIFT ? g * (TPR * NV + 1) + t : threadIdx.x) * 16, t4 = S::STATS + threadIdx.x * 4;
  const uint32_t fac = base + RING * SB + t * 16;
  int64_t row = blockIdx.x + (int64_t)gridDim.x * g;  // few rows spread over all SMs
  const bool has_x = p.g1 != nullptr || p.gate != nullptr;
  const uint8_t* dyp = static_cast<const uint8_t*>(p.dy) + row * p.lddy * ES + t * 16;
  const uint8_t* hp = static_cast<const uint8_t*>(p.h) + row * p.ldh * ES + t * 16;
  const uint8_t* dhp = static_cast<const uint8_t*>(p.dh) + row * p.lddh * ES + t * 16;
  const uint8_t* xp = static_cast<const uint8_t*>(p.x) + row * p.ldx * ES + t * 16;
  auto issue = [&](int64_t r, uint32_t slot) {
    if (r < p.M) {
      if (p.g2) {
        cp4(slot + t4, p.rs2 + r);
        if (FULL && p.layer) cp4(slot + t4 + 8 * T, p.mu2 + r);
      }
      if (p.g1) {
        cp4(slot + t4 + 4 * T, p.rs1 + r);
        if (FULL && p.layer) cp4(slot + t4 + 12 * T, p.mu1 + r);
      }
      if constexpr (SHIFT) {
        const uint32_t at = slot + t16 - t * 16;
        if (p.g2) {
          copy_row<TPR, NV>(at, dyp - t * 16, p.D * ES, t);
          copy_row<TPR, NV>(at + TB, hp - t * 16, p.D * ES, t);
        }
        if (p.dh) copy_row<TPR, NV>(at + 2 * TB, dhp - t * 16, p.D * ES, t);
        if (has_x) copy_row<TPR, NV>(at + 3 * TB, xp - t * 16, p.D * ES, t);
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if ((t + TPR * j) * EPC < p.D) {
            if (p.g2) {
              cp16(slot + t16 + j * WB, dyp + TPR * j * 16);
              cp16(slot + t16 + TB + j * WB, hp + TPR * j * 16);
            }
            if (p.dh) cp16(slot + t16 + 2 * TB + j * WB, dhp + TPR * j * 16);
            if (has_x) cp16(slot + t16 + 3 * TB + j * WB, xp + TPR * j * 16);
          }
        }
      }
      dyp += p.dystep;
      hp += p.hstep;
      dhp += p.dhstep;
      xp += p.xstep;
    }
    cp_commit();
  };
  // words past D, tensors and statistics that are not there hold zeros
#pragma unroll
  for (int k = 0; k < RING; ++k) {
#pragma unroll
    for (int i = 0; i < (FULL ? 4 : 2); ++i) sts4(base + k * SB + t4 + 4 * i * T, 0u);
#pragma unroll
    for (int j = 0; j < (SHIFT ? 0 : NV); ++j) {
      const bool in = (t + TPR * j) * EPC < p.D;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!in || !(i < 2 ? p.g2 != nullptr : i == 2 ? p.dh != nullptr : has_x)) sts16_zero(base + k * SB + t16 + i * TB + j * WB);
    }
  }
  // A thread's copies are not ordered behind its own stores, and they fill the statistics' slots that are zeroed above: they start
  // behind a barrier. (Zeroing only the slots that none fills spills 12 bytes in 256 threads of 32 columns: 4096 x 8192 94 -> 103 us.)
  __syncthreads();
#pragma unroll
  for (int k = 0; k < P; ++k) issue(row + k * p.step, base + k * SB);
  const DropKey key = drop_key(p.drop);
  uint4* fput = ring + RING * SB / 16;
  if (p.g2) put_factors<T, TPR, NV, EPC>(fput, 0, p.g2, nullptr, p.param_elem, 1.f, 0.f, p.D);
  put_factors<T, TPR, NV, EPC>(fput, 1, p.gate, p.g1, p.param_elem, p.scale, 1.f, p.D);
  __syncthreads();
  constexpr int NS = FULL ? 4 : 2;
  uint64_t acc[NS][NV][PP];  // sums of dy hhat, drop(dH) xhat, dy, drop(dH)
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < PP; ++k) acc[i][j][k] = 0;
  const float inv_d = 1.0f / (float)p.D;
  int turn = 0;
  uint32_t slot = base, last = base + P * SB;
  uint8_t* op = static_cast<uint8_t*>(p.dx) + row * p.lddx * ES + t * 16;
  uint8_t* drp = static_cast<uint8_t*>(p.dres) + row * p.lddres * ES + t * 16;
  // -mean(q xhat) and -mean(q), times the reciprocal deviation
  auto means = [&](uint64_t a1, uint64_t a2, float rs, uint64_t& m1, uint64_t& m2) {
    const float2 p2 = upk(a2);
    const float f = -inv_d * rs;
    if constexpr (FULL) {
      const float2 p1 = upk(a1);
      const float2 sums = row_sum2<TPR>(p1.x + p1.y, p2.x + p2.y, xch, turn);
      const float v = p.layer ? sums.x * f : 0.f;
      m1 = pk(v, v);
      m2 = pk(sums.y * f, sums.y * f);
    } else {
      const float v = row_sum<TPR>(p2.x + p2.y, xch, turn) * f;
      m1 = 0;
      m2 = pk(v, v);
    }
  };
  // word j of tensor i (0 dy, 1 h, 2 dh, 3 x) of the row in `slot`
  auto take = [&](uint32_t slot, int i, int j, const void* src, int64_t ld, uint64_t* v) {
    if constexpr (!SHIFT) {
      unpack_word<ELEM>(lds16(slot + t16 + i * TB + j * WB), v);
    } else if (src) {
      read_shifted<ELEM>(slot + t16 + i * TB + j * WB, row_shift(static_cast<const uint8_t*>(src) + row * ld * ES), (t + TPR * j) * EPC, p.D, v);
    } else {
#pragma unroll
      for (int k = 0; k < PP; ++k) v[k] = 0;
    }
  };
  // a normalised word, tensor 1 (h) or 3 (x)
  auto normal = [&](uint32_t slot, int i, int j, uint64_t rs2, uint64_t mu2, uint64_t* v) {
    take(slot, i, j, i == 1 ? p.h : p.x, i == 1 ? p.ldh : p.ldx, v);
#pragma unroll
    for (int k = 0; k < PP; ++k) {
      if constexpr (FULL) v[k] = sub_2(v[k], mu2);
      v[k] = mul_2(v[k], rs2);
    }
  };
  // groups of whole warps leave when they have no more rows; narrower ones go on while another of their warp has
  constexpr bool LEAVE = TPR >= 32;
  for (int64_t row0 = blockIdx.x; LEAVE ? row < p.M : row0 < p.M; row0 += p.step, row += p.step) {
    if constexpr (SHIFT) {
      cp_wait<P - 1>();
      group_meet<TPR>();  // the row is there for all, and all have left the slot that is filled next
      issue(row + P * p.step, last);
    } else {
      issue(row + P * p.step, last);
      cp_wait<P>();
    }
    const bool active = LEAVE || row < p.M;
    uint64_t d[NV][PP], xh[REMAKE ? 1 : NV][PP];
    uint32_t draws[NV][PP];  // drawn ahead of the sums, beside whose exchanges they cost least
    if (p.drop.cut) {
#pragma unroll
      for (int j = 0; j < NV; ++j) word_draws<EPC, SHIFT>(key, (t + TPR * j) * EPC, p.D, (uint32_t)row, draws[j]);
    }
    uint64_t rs2 = 0, mu2 = 0, m1 = 0, m2 = 0;
    if (p.g2) {
      const float rs = __uint_as_float(lds4(slot + t4)), mu = FULL ? __uint_as_float(lds4(slot + t4 + 8 * T)) : 0.f;
      rs2 = pk(rs, rs);
      mu2 = pk(mu, mu);
      uint64_t a1 = 0, a2 = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        uint64_t f[PP];
        get_factors<TPR, NV, EPC>(fac, 0, j, f);
        uint64_t* v = xh[REMAKE ? 0 : j];
        take(slot, 0, j, p.dy, p.lddy, d[j]);
        take(slot, 1, j, p.h, p.ldh, v);
#pragma unroll
        for (int k = 0; k < PP; ++k) {
          if constexpr (FULL) v[k] = sub_2(v[k], mu2);
          v[k] = mul_2(v[k], rs2);
          if (active) {
            acc[0][j][k] = fma_2(d[j][k], v[k], acc[0][j][k]);
            if constexpr (FULL) acc[2][j][k] = add_2(acc[2][j][k], d[j][k]);
          }
          d[j][k] = mul_2(d[j][k], f[k]);  // zero past D
          if constexpr (FULL) a1 = add_2(a1, d[j][k]);
          a2 = fma_2(d[j][k], v[k], a2);
        }
      }
      means(a1, a2, rs, m1, m2);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < PP; ++k) d[j][k] = xh[REMAKE ? 0 : j][k] = 0;
    }
    const float rs = __uint_as_float(lds4(slot + t4 + 4 * T)), mu = FULL ? __uint_as_float(lds4(slot + t4 + 12 * T)) : 0.f;
    const uint64_t rs1 = p.g1 ? pk(rs, rs) : pk(1.f, 1.f), mu1 = pk(mu, mu);
    uint64_t a1 = 0, a2 = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t r[PP], *v = xh[REMAKE ? 0 : j];
      take(slot, 2, j, p.dh, p.lddh, r);
      if constexpr (REMAKE) normal(slot, 1, j, rs2, mu2, v);
#pragma unroll
      for (int k = 0; k < PP; ++k) {  // dH
        if constexpr (FULL) r[k] = add_2(r[k], m1);
        d[j][k] = fma_2(v[k], m2, fma_2(d[j][k], rs2, r[k]));
      }
      if constexpr (SHIFT) {
        if (p.dres) write_shifted<ELEM, TPR>(drp - t * 16, (t + TPR * j) * EPC, p.D, t, active, pack_word<ELEM>(d[j]));
      } else if (p.dres && active && (t + TPR * j) * EPC < p.D) {
        *reinterpret_cast<uint4*>(drp + TPR * j * 16) = pack_word<ELEM>(d[j]);
      }
      if (p.drop.cut) {
#pragma unroll
        for (int k = 0; k < PP; ++k) d[j][k] = drop_pair(d[j][k], draws[j][k], key.cutw);
      }
      uint64_t f[PP];
      get_factors<TPR, NV, EPC>(fac, 1, j, f);  // zeros past D
      if (has_x) {
        take(slot, 3, j, p.x, p.ldx, v);
#pragma unroll
        for (int k = 0; k < PP; ++k) {
          if constexpr (FULL) v[k] = sub_2(v[k], mu1);
          v[k] = mul_2(v[k], rs1);
          if (active) {
            acc[1][j][k] = fma_2(d[j][k], v[k], acc[1][j][k]);
            if constexpr (FULL) acc[3][j][k] = add_2(acc[3][j][k], d[j][k]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < PP; ++k) {
        d[j][k] = mul_2(d[j][k], f[k]);
        if constexpr (FULL) a1 = add_2(a1, d[j][k]);
        a2 = fma_2(d[j][k], v[k], a2);
      }
    }
    if (p.g1) {
      means(a1, a2, rs, m1, m2);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        uint64_t* v = xh[REMAKE ? 0 : j];
        if constexpr (REMAKE) normal(slot, 3, j, rs1, mu1, v);
#pragma unroll
        for (int k = 0; k < PP; ++k) {
          uint64_t o = mul_2(v[k], m2);
          if constexpr (FULL) o = add_2(o, m1);
          d[j][k] = fma_2(d[j][k], rs1, o);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (SHIFT) write_shifted<ELEM, TPR>(op - t * 16, (t + TPR * j) * EPC, p.D, t, active, pack_word<ELEM>(d[j]));
      else if (active && (t + TPR * j) * EPC < p.D) *reinterpret_cast<uint4*>(op + TPR * j * 16) = pack_word<ELEM>(d[j]);
    }
    op += p.dxstep;
    drp += p.drstep;
    last = slot;
    slot = slot == base + P * SB ? base : slot + SB;
  }
  cp_wait<0>();
  // column partials: the row groups of a warp by shuffles, then the others' over the ring's memory, a column's in the groups' order
  float* red = reinterpret_cast<float*>(ring);
  constexpr int TURNS = TPR < 32 ? T / 32 : GPB, COLS = TPR * NV * EPC;
  static_assert(S::SMEM >= (size_t)TURNS * COLS * sizeof(float), "the column partials reuse the ring");
  if constexpr (TPR < 32) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < PP; ++k)
#pragma unroll
          for (int o = TPR; o < 32; o <<= 1) acc[i][j][k] = add_2(acc[i][j][k], __shfl_xor_sync(0xFFFFFFFFu, acc[i][j][k], o));
  }
  const int mine = TPR < 32 ? (int)threadIdx.x >> 5 : g;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    constexpr int kPlace[4] = {0, 2, 1, 3};
    if (!(p.sums >> kPlace[i] & 1)) continue;
    float* part = p.part + ((int64_t)blockIdx.x * 4 + kPlace[i]) * p.D;
    __syncthreads();  // the ring, or the sum before this one, has been read
    if (TPR >= 32 || (threadIdx.x & 31) < TPR) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < PP / 2; ++q) {
          const float2 lo = upk(acc[i][j][2 * q]), hi = upk(acc[i][j][2 * q + 1]);
          *reinterpret_cast<float4*>(red + mine * COLS + (t + TPR * j) * EPC + 4 * q) = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += T) {
      float v = red[c];
#pragma unroll
      for (int q = 1; q < TURNS; ++q) v += red[q * COLS + c];
      part[c] = v;
    }
  }
}

// ------------------------------------------------------------ 16-bit rows of 8200 to 16384 columns
// A block's 512 threads share a row, 32 columns each. The registers hold the sums of dy hhat and dt xhat and the gradient on its
// way down; the normalised values are made again from the row's words in shared memory for each pass over them, and the sums for the betas
// (FULL) live in shared memory too, where dh then has no place and is loaded behind the first pass. A tensor's words of the next row
// are copied once the last pass over them is done. 2048 x 16384 bf16 119 us, 51% of a copy
// (by single elements 348), with layer norms, betas and a gate 155 (371).
template <int ELEM, bool FULL>
struct JoinBwdWide {
  static constexpr int T = 512, NV = 4, EPC = Word<ELEM>::EPC, TENSOR = NV * T * 16, TENSORS = FULL ? 3 : 4;  // dy, h, x, dh
  static constexpr int SUMS = FULL ? 2 * T * NV * EPC * 4 : 0;
  static constexpr size_t SMEM = TENSORS * TENSOR + SUMS;
  static_assert(SMEM <= kVecSmem && EPC == 8, "shared memory budget");
};
template <int ELEM, bool FULL>
__global__ void __launch_bounds__(512, 1) join_bwd_wide_kernel(const JoinBwdParams p) {
  using S = JoinBwdWide<ELEM, FULL>;
  constexpr int T = S::T, NV = S::NV, EPC = S::EPC, PP = EPC / 2;
  constexpr uint32_t WB = T * 16, TB = S::TENSOR;
  __shared__ float2 xch[2 * T / 32];
  extern __shared__ uint4 ring[];  // [TENSORS][NV][T], then the sums of dy and dt, [2][2 NV quarters of 8][T] float4
  const int t = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(ring) + t * 16;
  float4* sums = reinterpret_cast<float4*>(ring + S::TENSORS * TB / 16) + t;
  const bool has_x = p.g1 != nullptr || p.gate != nullptr;
  auto col = [&](int j) { return (t + T * j) * EPC; };
  auto copy = [&](int i, const void* src, int64_t ld, int64_t row) {
    const uint8_t* r = static_cast<const uint8_t*>(src) + row * ld * 2 + t * 16;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (col(j) < p.D) cp16(at + i * TB + j * WB, r + j * T * 16);
  };
  auto copy_first = [&](int64_t row) {  // what the first pass reads
    if (row < p.M && p.g2) {
      copy(0, p.dy, p.lddy, row);
      copy(1, p.h, p.ldh, row);
    }
    cp_commit();
  };
  auto copy_second = [&](int64_t row) {
    if (row < p.M) {
      if (has_x) copy(2, p.x, p.ldx, row);
      if constexpr (!FULL)
        if (p.dh) copy(3, p.dh, p.lddh, row);
    }
    cp_commit();
  };
  // words past D and tensors that are not there hold zeros
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < S::TENSORS; ++i)
      if (col(j) >= p.D || !(i < 2 ? p.g2 != nullptr : i == 2 ? has_x : p.dh != nullptr)) sts16_zero(at + i * TB + j * WB);
    if constexpr (FULL)
#pragma unroll
      for (int q = 0; q < 4; ++q) sums[(4 * j + q) * T] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  copy_first(blockIdx.x);
  copy_second(blockIdx.x);
  const DropKey key = drop_key(p.drop);
  uint64_t acc[2][NV][PP];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < PP; ++k) acc[i][j][k] = 0;
  auto add_sums = [&](int which, int j, const uint64_t* v) {  // to the sums of dy (0) or dt (1)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float4* s = sums + (which * 2 * NV + 2 * j + q) * T;
      const float2 a = upk(v[2 * q]), b = upk(v[2 * q + 1]);
      const float4 o = *s;
      *s = make_float4(o.x + a.x, o.y + a.y, o.z + b.x, o.w + b.y);
    }
  };
  const float inv_d = 1.0f / (float)p.D;
  int turn = 0;
  auto means = [&](uint64_t a1, uint64_t a2, float rs, uint64_t& m1, uint64_t& m2) {
    const float2 p2 = upk(a2);
    const float f = -inv_d * rs;
    if constexpr (FULL) {
      const float2 p1 = upk(a1);
      const float2 s = row_sum2<T>(p1.x + p1.y, p2.x + p2.y, xch, turn);
      const float v = p.layer ? s.x * f : 0.f;
      m1 = pk(v, v);
      m2 = pk(s.y * f, s.y * f);
    } else {
      const float v = row_sum<T>(p2.x + p2.y, xch, turn) * f;
      m1 = 0;
      m2 = pk(v, v);
    }
  };
  // a normalised word, tensor 1 (h) or 2 (x)
  auto normal = [&](int i, int j, uint64_t rs2, uint64_t mu2, uint64_t* v) {
    unpack_word<ELEM>(lds16(at + i * TB + j * WB), v);
#pragma unroll
    for (int k = 0; k < PP; ++k) {
      if constexpr (FULL) v[k] = sub_2(v[k], mu2);
      v[k] = mul_2(v[k], rs2);
    }
  };
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const float rsb = p.g2 ? p.rs2[row] : 0.f, rsa = p.g1 ? p.rs1[row] : 1.f;
    const float mub = FULL && p.layer && p.g2 ? p.mu2[row] : 0.f, mua = FULL && p.layer && p.g1 ? p.mu1[row] : 0.f;
    const uint64_t rs2 = pk(rsb, rsb), mu2 = pk(mub, mub), rs1 = pk(rsa, rsa), mu1 = pk(mua, mua);
    cp_wait<1>();
    uint64_t a1 = 0, a2 = 0, m1 = 0, m2 = 0;
    uint4 dhw[FULL ? NV : 1];
    if (p.g2) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        uint64_t f[PP], q[PP], xh[PP];
        load_params<EPC>(p.g2, p.param_elem, col(j) < p.D ? col(j) : 0, f);
        unpack_word<ELEM>(lds16(at + j * WB), q);
        normal(1, j, rs2, mu2, xh);
        if constexpr (FULL) add_sums(0, j, q);
#pragma unroll
        for (int k = 0; k < PP; ++k) {
          acc[0][j][k] = fma_2(q[k], xh[k], acc[0][j][k]);
          q[k] = mul_2(q[k], f[k]);  // zero past D
          if constexpr (FULL) a1 = add_2(a1, q[k]);
          a2 = fma_2(q[k], xh[k], a2);
        }
      }
    }
    if constexpr (FULL) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        dhw[j] = make_uint4(0u, 0u, 0u, 0u);
        if (p.dh && col(j) < p.D) dhw[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dh) + row * p.lddh + col(j));
      }
    }
    if (p.g2) means(a1, a2, rsb, m1, m2);
    cp_wait<0>();
    uint64_t d[NV][PP];
    a1 = a2 = 0;
    uint16_t* dr = static_cast<uint16_t*>(p.dres) + row * p.lddres;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = col(j) < p.D;
      const int c = in ? col(j) : 0;
      uint64_t xh[PP], f[PP], g[PP];
      unpack_word<ELEM>(lds16(at + j * WB), d[j]);
      normal(1, j, rs2, mu2, xh);
      params_or<EPC>(p.g2, p.param_elem, c, 0.f, f);
      if constexpr (FULL) unpack_word<ELEM>(dhw[j], g);
      else unpack_word<ELEM>(lds16(at + 3 * TB + j * WB), g);
#pragma unroll
      for (int k = 0; k < PP; ++k) {  // dH
        if constexpr (FULL) g[k] = add_2(g[k], m1);
        d[j][k] = fma_2(xh[k], m2, fma_2(mul_2(d[j][k], f[k]), rs2, g[k]));
      }
      if (p.dres && in) *reinterpret_cast<uint4*>(dr + c) = pack_word<ELEM>(d[j]);
      if (p.drop.cut) {
        uint32_t draws[PP];
        word_draws<EPC>(key, c, p.D, (uint32_t)row, draws);
#pragma unroll
        for (int k = 0; k < PP; ++k) d[j][k] = drop_pair(d[j][k], draws[k], key.cutw);
      }
      normal(2, j, rs1, mu1, xh);
#pragma unroll
      for (int k = 0; k < PP; ++k) acc[1][j][k] = fma_2(d[j][k], xh[k], acc[1][j][k]);
      if constexpr (FULL) add_sums(1, j, d[j]);
      params_or<EPC>(p.gate, p.param_elem, c, 1.f, f);
      params_or<EPC>(p.g1, p.param_elem, c, 1.f, g);
#pragma unroll
      for (int k = 0; k < PP; ++k) {
        d[j][k] = in ? mul_2(d[j][k], mul_2(mul_2(f[k], pk(p.scale, p.scale)), g[k])) : 0;
        if constexpr (FULL) a1 = add_2(a1, d[j][k]);
        a2 = fma_2(d[j][k], xh[k], a2);
      }
    }
    copy_first(row + gridDim.x);
    if (p.g1) means(a1, a2, rsa, m1, m2);
    uint16_t* o = static_cast<uint16_t*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (p.g1) {
        uint64_t xh[PP];
        normal(2, j, rs1, mu1, xh);
#pragma unroll
        for (int k = 0; k < PP; ++k) {
          uint64_t v = mul_2(xh[k], m2);
          if constexpr (FULL) v = add_2(v, m1);
          d[j][k] = fma_2(d[j][k], rs1, v);
        }
      }
      if (col(j) < p.D) *reinterpret_cast<uint4*>(o + col(j)) = pack_word<ELEM>(d[j]);
    }
    copy_second(row + gridDim.x);
  }
  cp_wait<0>();
  // a column is one thread's: its sums are the block's
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // the places of `part`: dy hhat, dy, dt xhat, dt
    if (!(p.sums >> i & 1)) continue;
    float* part = p.part + ((int64_t)blockIdx.x * 4 + i) * p.D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (col(j) >= p.D) continue;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float4 v;
        if (i == 0 || i == 2) {
          const float2 a = upk(acc[i / 2][j][2 * q]), b = upk(acc[i / 2][j][2 * q + 1]);
          v = make_float4(a.x, a.y, b.x, b.y);
        } else {
          v = FULL ? sums[((i / 2) * 2 * NV + 2 * j + q) * T] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        *reinterpret_cast<float4*>(part + col(j) + 4 * q) = v;
      }
    }
  }
}

// The column sums of n partial rows in a fixed order (32 columns a block, warp w adds rows w, w + 32, ..., then the warps'
// sums are added over the lanes), and what the gradients make of them: blocks y = 0 those of the second norm, y = 1 of the first
// and the gate. A few hundred rows are all latency: both sums' loads of five rows a warp, all that an SM's one block leaves, are on
// their way together.
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
  float scale;  // of the last two sums
};
__global__ void __launch_bounds__(1024) join_sum_kernel(const JoinSumParams p) {
  __shared__ float red[2][32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, cw = blockIdx.x * 32 + w;
  const int first = 2 * blockIdx.y;  // of this block's two sums
  const bool has[2] = {(p.sums >> first & 1) != 0, (p.sums >> first & 2) != 0};
  float s[2] = {0.f, 0.f};
  for (int i0 = w; i0 < p.n; i0 += 32 * 5) {
    float v[2][5];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        const int i = i0 + 32 * u;
        v[k][u] = has[k] && c < p.D && i < p.n ? __ldcs(p.part + ((int64_t)i * 4 + first + k) * p.D + c) : 0.f;
      }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int u = 0; u < 5; ++u) s[k] += v[k][u];
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) red[k][w][lane] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) s[k] = warp_sum(red[k][lane][w]);  // warp w: column w of the block
  if (lane != 0 || cw >= p.D) return;
  if (blockIdx.y == 0) {
    if (p.dg2) p.dg2[cw] = s[0];
    if (p.db2) p.db2[cw] = s[1];
    return;
  }
  const float f = param_or(p.gate, p.param_elem, cw, 1.f);
  s[0] *= p.scale;
  s[1] *= p.scale;
  if (p.dg1) p.dg1[cw] = f * s[0];
  if (p.db1) p.db1[cw] = f * s[1];
  if (p.dgate) p.dgate[cw] = p.g1 ? fmaf(load_elem_rt(p.g1, p.param_elem, cw), s[0], p.b1 ? load_elem_rt(p.b1, p.param_elem, cw) * s[1] : 0.f) : s[0];
}

// ------------------------------------------------------------ host side
constexpr int kBwdBlocksPerSm = 2;  // at most: each leaves partial rows of the column sums

template <int ELEM, int TPR, int NE>
lnfp8_status bwd_any_launch(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  constexpr auto kernel = join_bwd_any_kernel<ELEM, TPR, NE>;
  constexpr int threads = TPR < 256 ? 256 : TPR, gpb = threads / TPR;
  constexpr size_t smem = TPR >= 1024 ? 3 * TPR * NE * sizeof(float) : gpb > 1 ? TPR * NE * sizeof(float) : 0;
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
  if constexpr (ELEM == LNFP8_FP32) {
    if (p.D <= 256) return bwd_any_launch<ELEM, 32, 8>(p, blocks_out, st);
    if (p.D <= 512) return bwd_any_launch<ELEM, 64, 8>(p, blocks_out, st);
    if (p.D <= 1024) return bwd_any_launch<ELEM, 128, 8>(p, blocks_out, st);
    if (p.D <= 2048) return bwd_any_launch<ELEM, 256, 8>(p, blocks_out, st);
    if (p.D <= 4096) return bwd_any_launch<ELEM, 512, 8>(p, blocks_out, st);
    if (p.D <= 8192) return bwd_any_launch<ELEM, 1024, 8>(p, blocks_out, st);
  }
  return bwd_any_launch<ELEM, 1024, 16>(p, blocks_out, st);
}

// Threads of a block (one an SM): as many as leave each the registers of its sums and its row: 256 for 24 columns of four sums or
// 32 whose normalised values are made again, 384 for 16 of four or 24 of two, 512 for less; groups of 96, 192 and 384 threads
// fill 384.
constexpr int bwd_threads(int elem, int tpr, int nv, bool full) {
  if (nv >= 3) return full || tpr == 256 ? 256 : 384;
  if (tpr % 96 == 0) return 384;
  return full && elem != LNFP8_FP32 && tpr <= 128 ? 384 : 512;
}
template <int ELEM, int TPR, int NV, bool FULL, bool SHIFT = false>
lnfp8_status bwd_vec_launch(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  constexpr int T = bwd_threads(ELEM, TPR, NV, FULL);
  using S = JoinBwdShape<ELEM, TPR, NV, FULL, T, SHIFT>;
  constexpr auto kernel = join_bwd_vec_kernel<ELEM, TPR, NV, FULL, T, SHIFT>;
  const lnfp8_status s = kernel_setup<kernel>(T, S::SMEM, nullptr, "block_join_bwd: kernel set-up");
  if (s != LNFP8_OK) return s;
  constexpr int gpb = T / TPR, es = ElemSize<ELEM>::value;
  const int64_t blocks = min64(p.M, num_sms());
  *blocks_out = (int)blocks;
  JoinBwdParams q = p;
  q.step = blocks * gpb;
  q.dhstep = q.step * p.lddh * es;
  q.dystep = q.step * p.lddy * es;
  q.xstep = q.step * p.ldx * es;
  q.hstep = q.step * p.ldh * es;
  q.dxstep = q.step * p.lddx * es;
  q.drstep = q.step * p.lddres * es;
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(T), S::SMEM, st, q) != cudaSuccess) return check_launch("block_join_bwd launch");
  return check_launch("block_join_bwd");
}
// Columns a thread: 16 of a 16-bit type; 24 where those would leave a quarter of the threads or more without any (us, bf16:
// 16384 x 768 46 -> 38, 16384 x 2560 with two RMS norms and dropout 137 -> 103, with two layer norms, betas and a gate 218 -> 127, 8192 x
// 5120 148 -> 113 and 200 -> 128; groups of 192 and 384 threads of 16 columns 121, 150, 124 and 154); 32 with four sums, whose
// row then costs each SM fewer exchanges and whose registers hold nothing twice (two layer norms, betas and a gate, 32 and 16 columns:
// 65536 x 512 75 and 85, 16384 x 1024 44 and 53, 16384 x 2048 87 and 99, 8192 x 4096 91 and 119, 4096 x 8192 96 and 117; of two sums
// 32 columns gain up to 7% at 4096 and lose a fifth at 8192).
template <int ELEM, bool FULL>
lnfp8_status bwd_vec16(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  if (p.D <= 128) return bwd_vec_launch<ELEM, 8, 2, FULL>(p, blocks_out, st);
  if (p.D <= 256) return bwd_vec_launch<ELEM, 16, 2, FULL>(p, blocks_out, st);
  if (p.D <= 512) return bwd_vec_launch<ELEM, FULL ? 16 : 32, FULL ? 4 : 2, FULL>(p, blocks_out, st);
  if (p.D <= 32 * 24) return bwd_vec_launch<ELEM, 32, 3, FULL>(p, blocks_out, st);
  if (p.D <= 1024) return bwd_vec_launch<ELEM, FULL ? 32 : 64, FULL ? 4 : 2, FULL>(p, blocks_out, st);
  if (p.D <= 64 * 24) return bwd_vec_launch<ELEM, 64, 3, FULL>(p, blocks_out, st);
  if (p.D <= 2048) return bwd_vec_launch<ELEM, FULL ? 64 : 128, FULL ? 4 : 2, FULL>(p, blocks_out, st);
  if (p.D <= 128 * 24) return bwd_vec_launch<ELEM, 128, 3, FULL>(p, blocks_out, st);
  if (p.D <= 4096) return bwd_vec_launch<ELEM, FULL ? 128 : 256, FULL ? 4 : 2, FULL>(p, blocks_out, st);
  if (p.D <= 256 * 24) return bwd_vec_launch<ELEM, 256, 3, FULL>(p, blocks_out, st);
  return bwd_vec_launch<ELEM, FULL ? 256 : 512, FULL ? 4 : 2, FULL>(p, blocks_out, st);
}
// Of fp32 8 columns, whose words of four tensors fill the ring sooner, with groups of 96, 192 and 384 threads too (two layer norms
// and a gate: 8191 x 768 42 -> 37 us; with betas 8191 x 1280 75 -> 65, 8191 x 2560 154 -> 129).
template <bool FULL>
lnfp8_status bwd_vec32(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  constexpr int E = LNFP8_FP32;
  if (p.D <= 64) return bwd_vec_launch<E, 8, 2, FULL>(p, blocks_out, st);
  if (p.D <= 128) return bwd_vec_launch<E, 16, 2, FULL>(p, blocks_out, st);
  if (p.D <= 256) return bwd_vec_launch<E, 32, 2, FULL>(p, blocks_out, st);
  if (p.D <= 512) return bwd_vec_launch<E, 64, 2, FULL>(p, blocks_out, st);
  if (p.D <= 768) return bwd_vec_launch<E, 96, 2, FULL>(p, blocks_out, st);
  if (p.D <= 1024) return bwd_vec_launch<E, 128, 2, FULL>(p, blocks_out, st);
  if (p.D <= 1536) return bwd_vec_launch<E, 192, 2, FULL>(p, blocks_out, st);
  if (p.D <= 2048) return bwd_vec_launch<E, 256, 2, FULL>(p, blocks_out, st);
  if (p.D <= 384 * 8) return bwd_vec_launch<E, 384, 2, FULL>(p, blocks_out, st);
  return bwd_vec_launch<E, 512, 2, FULL>(p, blocks_out, st);
}
template <int ELEM, bool FULL>
lnfp8_status bwd_wide(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  using S = JoinBwdWide<ELEM, FULL>;
  constexpr auto kernel = join_bwd_wide_kernel<ELEM, FULL>;
  const lnfp8_status s = kernel_setup<kernel>(S::T, S::SMEM, nullptr, "block_join_bwd: kernel set-up");
  if (s != LNFP8_OK) return s;
  const int64_t blocks = min64(p.M, num_sms());
  *blocks_out = (int)blocks;
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(S::T), S::SMEM, st, p) != cudaSuccess) return check_launch("block_join_bwd launch");
  return check_launch("block_join_bwd");
}
template <int ELEM>
lnfp8_status bwd_shift(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  if (p.D <= 128) return bwd_vec_launch<ELEM, 8, 2, true, true>(p, blocks_out, st);
  if (p.D <= 256) return bwd_vec_launch<ELEM, 16, 2, true, true>(p, blocks_out, st);
  if (p.D <= 512) return bwd_vec_launch<ELEM, 32, 2, true, true>(p, blocks_out, st);
  if (p.D <= 1024) return bwd_vec_launch<ELEM, 64, 2, true, true>(p, blocks_out, st);
  if (p.D <= 2048) return bwd_vec_launch<ELEM, 128, 2, true, true>(p, blocks_out, st);
  if (p.D <= 4096) return bwd_vec_launch<ELEM, 256, 2, true, true>(p, blocks_out, st);
  return bwd_vec_launch<ELEM, 512, 2, true, true>(p, blocks_out, st);
}
// As the forward's.
template <int ELEM>
lnfp8_status bwd(const JoinBwdParams& p, int* blocks_out, cudaStream_t st) {
  constexpr int es = ElemSize<ELEM>::value;
  const bool wide = p.D > 1024 * Word<ELEM>::EPC;
  const bool vec = p.D % 8 == 0 && row_aligned(p.dx, p.lddx, es) && (!p.dres || row_aligned(p.dres, p.lddres, es)) &&
                   (!p.dh || row_aligned(p.dh, p.lddh, es)) && (!p.g2 || (row_aligned(p.dy, p.lddy, es) && row_aligned(p.h, p.ldh, es))) &&
                   (!(p.g1 || p.gate) || row_aligned(p.x, p.ldx, es)) && (!wide || vectors_aligned({p.g1, p.gate, p.g2}));
  const bool full = (p.layer && (p.g1 || p.g2)) || (p.sums & 10);
  if constexpr (ELEM == LNFP8_FP32) {
    if (!vec || wide) return bwd_any<ELEM>(p, blocks_out, st);
  } else {
    if (!vec) return wide ? bwd_any<ELEM>(p, blocks_out, st) : bwd_shift<ELEM>(p, blocks_out, st);
    if (wide) return full ? bwd_wide<ELEM, true>(p, blocks_out, st) : bwd_wide<ELEM, false>(p, blocks_out, st);
  }
  if constexpr (ELEM == LNFP8_FP32) return full ? bwd_vec32<true>(p, blocks_out, st) : bwd_vec32<false>(p, blocks_out, st);
  else return full ? bwd_vec16<ELEM, true>(p, blocks_out, st) : bwd_vec16<ELEM, false>(p, blocks_out, st);
}

}  // namespace

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
    s = a->elem == LNFP8_BF16   ? bwd<LNFP8_BF16>(p, &blocks, st)
        : a->elem == LNFP8_FP16 ? bwd<LNFP8_FP16>(p, &blocks, st)
                                : bwd<LNFP8_FP32>(p, &blocks, st);
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
  q.scale = p.scale;
  LaunchScope ls("block_join_sum", st);
  if (launch_pdl(join_sum_kernel, dim3((unsigned)((p.D + 31) / 32), 2), dim3(1024), 0, st, q) != cudaSuccess)
    return check_launch("block_join_bwd launch");
  return check_launch("block_join_bwd: column sums");
}

}  // namespace lnfp8
