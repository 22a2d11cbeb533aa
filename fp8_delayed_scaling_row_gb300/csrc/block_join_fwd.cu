// The forward of the join of a block's output with the residual stream (block_join.cuh).
#include "block_join.cuh"

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
  int64_t step, xstep, rstep, hstep, ystep;  // rows a group moves on by; the same in bytes of each tensor
};

template <int ELEM, int TPR, int NE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR <= 256 ? 2 : 1) join_fwd_any_kernel(const JoinFwdParams p) {
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
  constexpr bool HOLD = TPR <= 512;         // the columns' factors stay in registers
  float fa[HOLD ? NE : 1], fc[HOLD ? NE : 1], fg[HOLD ? NE : 1], fb[HOLD ? NE : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = tc + (i < n ? TPR * i : 0);
      const float f = p.scale * param_or(p.gate, p.param_elem, c, 1.f);
      fa[i] = f * param_or(p.g1, p.param_elem, c, 1.f);
      fc[i] = p.b1 ? f * param_or(p.b1, p.param_elem, c, 0.f) : 0.f;  // no beta: none of a gate that may be infinite
      fg[i] = param_or(p.g2, p.param_elem, c, 0.f);
      fb[i] = param_or(p.b2, p.param_elem, c, 0.f);
    }
  }
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
  // the bits of the next row, where there are registers for them, are on their way while one is worked on
  constexpr bool AHEAD = TPR <= 512;
  uint32_t xb[NE], rb[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) rb[i] = 0u;
  auto fetch = [&](int64_t row) {
    const int64_t rowc = min64(row, p.M - 1);
    const uint8_t* xr = static_cast<const uint8_t*>(p.x) + (rowc * p.ldx + tc) * ES;
    const uint8_t* rr = static_cast<const uint8_t*>(p.resid) + (rowc * p.ldr + tc) * ES;
#pragma unroll
    for (int i = 0; i < NE; ++i) xb[i] = load_bits<ELEM>(xr, i < n ? TPR * i : 0);
    if (p.resid) {
#pragma unroll
      for (int i = 0; i < NE; ++i) rb[i] = load_bits<ELEM>(rr, i < n ? TPR * i : 0);
    }
  };
  if constexpr (AHEAD) fetch((int64_t)blockIdx.x * GPB + g);
  for (int64_t row0 = (int64_t)blockIdx.x * GPB; row0 < p.M; row0 += (int64_t)gridDim.x * GPB) {
    const int64_t row = row0 + g;
    const bool active = row < p.M;
    if constexpr (!AHEAD) fetch(row);
    float v[NE], mu, rs;
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] = active && i < n ? bits_value<ELEM>(xb[i]) : 0.f;
    float r[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) r[i] = bits_value<ELEM>(rb[i]);
    if constexpr (AHEAD) fetch(row + (int64_t)gridDim.x * GPB);
    if (p.g1) {
      normalise(v, mu, rs);
      if (t == 0 && active) {
        p.rs1[row] = rs;
        if (p.layer) p.mu1[row] = mu;
      }
    }
    if (p.drop.cut) any_draws<NE>(bits, key, t, TPR, (uint32_t)row);
    if constexpr (HOLD) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = fmaf(v[i], fa[i], fc[i]);
    } else {  // one vector after the other
      float f[NE];
      if (p.g1) {
        load_params_any<TPR, NE>(p.g1, p.param_elem, tc, n, f);
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] *= f[i];
      }
      if (p.b1) {
        load_params_any<TPR, NE>(p.b1, p.param_elem, tc, n, f);
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] += f[i];
      }
      if (p.gate) {
        load_params_any<TPR, NE>(p.gate, p.param_elem, tc, n, f);
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] *= f[i];
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] *= p.scale;
    }
    uint8_t* hr = static_cast<uint8_t*>(p.h) + (row * p.ldh + t) * ES;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const bool keep = p.drop.cut == 0 || bits[32 * i + lane] >= p.drop.cut;
      const float sum = r[i] + (keep ? v[i] : 0.f);
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
    if constexpr (HOLD) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = fmaf(v[i], fg[i], fb[i]);
    } else {
      float f[NE];
      load_params_any<TPR, NE>(p.g2, p.param_elem, tc, n, f);
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] *= f[i];
      if (p.b2) {
        load_params_any<TPR, NE>(p.b2, p.param_elem, tc, n, f);
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] += f[i];
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i < n) store_elem<ELEM>(yr, TPR * i, v[i]);
  }
}

template <int ELEM, int TPR, int NV, bool FULL, bool SHIFT>
struct JoinFwdShape {
  // bytes of a tensor's rows (x, residual): words of all threads, with SHIFT one more a row
  static constexpr int TENSOR = (kVecThreads * NV + (SHIFT ? kVecThreads / TPR : 0)) * 16;
  // Rows of more than 8192 columns: the factors would not fit beside two rows and are made of the vectors for each row.
  static constexpr bool MAKE = TPR * NV * Word<ELEM>::EPC > 8192;
  static constexpr int SLOT = 2 * TENSOR, FACTORS = MAKE ? 0 : (FULL ? 4 : 2) * TPR * NV * Word<ELEM>::EPC * 4;
  static constexpr int FIT = (kVecSmem - FACTORS) / SLOT, RING = FIT < 4 ? FIT : 4;
  static constexpr size_t SMEM = (size_t)RING * SLOT + FACTORS;
  static_assert(RING >= 2, "shared memory budget");
};

template <int ELEM, int TPR, int NV, bool FULL, bool SHIFT>
__global__ void __launch_bounds__(kVecThreads, 1) join_fwd_vec_kernel(const JoinFwdParams p) {
  using S = JoinFwdShape<ELEM, TPR, NV, FULL, SHIFT>;
  constexpr int T = kVecThreads, RING = S::RING, P = RING - 1;
  constexpr int EPC = Word<ELEM>::EPC, PP = EPC / 2, ES = ElemSize<ELEM>::value;
  __shared__ float2 xch[2 * T / 32];
  // [RING][2 tensors][NV][T] (SHIFT: [2 tensors][groups][words of a row]), then the factors: gate post_gamma, pre_gamma,
  // gate post_beta, pre_beta (the scale is left to the sum with the residual, which then rounds once)
  extern __shared__ uint4 ring[];
  const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
  pdl_wait();
  pdl_launch_dependents();
  constexpr uint32_t WB = SHIFT ? TPR * 16 : T * 16, TB = S::TENSOR, SB = S::SLOT;  // bytes to a thread's next word, of a tensor, of a slot
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + (SHIFT ? g * (TPR * NV + 1) + t : threadIdx.x) * 16;
  const uint32_t fac = (uint32_t)__cvta_generic_to_shared(ring) + RING * SB + t * 16;
  int64_t row = blockIdx.x + (int64_t)gridDim.x * g;  // few rows spread over all SMs
  const uint8_t* xp = static_cast<const uint8_t*>(p.x) + row * p.ldx * ES + t * 16;
  const uint8_t* rp = static_cast<const uint8_t*>(p.resid) + row * p.ldr * ES + t * 16;
  auto issue = [&](int64_t r, uint32_t slot) {
    if (r < p.M) {
      if constexpr (SHIFT) {
        copy_row<TPR, NV>(slot - t * 16, xp - t * 16, p.D * ES, t);
        if (p.resid) copy_row<TPR, NV>(slot + TB - t * 16, rp - t * 16, p.D * ES, t);
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if ((t + TPR * j) * EPC < p.D) {
            cp16(slot + j * WB, xp + TPR * j * 16);
            if (p.resid) cp16(slot + TB + j * WB, rp + TPR * j * 16);
          }
        }
      }
      xp += p.xstep;
      rp += p.rstep;
    }
    cp_commit();
  };
  // words past D, and a residual that is not there, hold zeros
  if constexpr (!SHIFT) {
#pragma unroll
    for (int k = 0; k < RING; ++k)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const bool in = (t + TPR * j) * EPC < p.D;
        if (!in) sts16_zero(mine + k * SB + j * WB);
        if (!in || !p.resid) sts16_zero(mine + k * SB + TB + j * WB);
      }
  }
#pragma unroll
  for (int k = 0; k < P; ++k) issue(row + k * p.step, mine + k * SB);
  drop_save(p.drop);
  const DropKey key = drop_key(p.drop);
  if constexpr (!S::MAKE) {
    uint4* fput = ring + RING * SB / 16;
    put_factors<T, TPR, NV, EPC>(fput, 0, p.gate, p.g1, p.param_elem, 1.f, 1.f, p.D);
    if (p.g2) put_factors<T, TPR, NV, EPC>(fput, 1, p.g2, nullptr, p.param_elem, 1.f, 0.f, p.D);
    if constexpr (FULL) {
      put_factors<T, TPR, NV, EPC>(fput, 2, p.b1, p.b1 ? p.gate : nullptr, p.param_elem, 1.f, 0.f, p.D);  // no beta: none of a gate that may be infinite
      put_factors<T, TPR, NV, EPC>(fput, 3, p.b2, nullptr, p.param_elem, 1.f, 0.f, p.D);
    }
    __syncthreads();
  }
  // factor array k's part of word j, zeros past D
  auto factors = [&](int k, int j, uint64_t* f) {
    if constexpr (!S::MAKE) {
      get_factors<TPR, NV, EPC>(fac, k, j, f);
    } else {
      const int c = (t + TPR * j) * EPC, cc = c < p.D ? c : 0;
      params_or<EPC>(k == 0 ? p.g1 : k == 1 ? p.g2 : k == 2 ? p.b1 : p.b2, p.param_elem, cc, k == 0 ? 1.f : 0.f, f);
      if (k == 0 || (k == 2 && p.b1)) {
        uint64_t a[PP];
        params_or<EPC>(p.gate, p.param_elem, cc, 1.f, a);
#pragma unroll
        for (int i = 0; i < PP; ++i) f[i] = mul_2(a[i], f[i]);
      }
      if (c >= p.D) {
#pragma unroll
        for (int i = 0; i < PP; ++i) f[i] = 0;
      }
    }
  };
  const float inv_d = 1.0f / (float)p.D;
  const uint64_t scale2 = pk(p.scale, p.scale);
  int turn = 0;
  uint32_t slot = mine, last = mine + P * SB;  // the row's slot; the one read before it, filled next
  uint8_t* hp = static_cast<uint8_t*>(p.h) + row * p.ldh * ES + t * 16;
  uint8_t* yp = static_cast<uint8_t*>(p.y) + row * p.ldy * ES + t * 16;
  // v becomes the centred row (FULL); returns the reciprocal deviation
  auto stats = [&](uint64_t(&v)[NV][PP], float& mu) {
    mu = 0.f;
    if (FULL && p.layer) {
      uint64_t s2 = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < PP; ++k) s2 = add_2(s2, v[j][k]);
      const float2 s = upk(s2);
      mu = row_sum<TPR>(s.x + s.y, xch, turn) * inv_d;
      const uint64_t mu2 = pk(mu, mu);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (t + TPR * j) * EPC;
        if (c >= p.D) continue;
#pragma unroll
        for (int k = 0; k < PP; ++k) v[j][k] = sub_2(v[j][k], mu2);
        if (SHIFT && c + EPC > p.D) {
#pragma unroll
          for (int k = 0; k < PP; ++k) {
            const float2 f = upk(v[j][k]);
            v[j][k] = pk(c + 2 * k < p.D ? f.x : 0.f, c + 2 * k + 1 < p.D ? f.y : 0.f);
          }
        }
      }
    }
    uint64_t q2 = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < PP; ++k) q2 = fma_2(v[j][k], v[j][k], q2);
    const float2 q = upk(q2);
    return rsqrt_nr(row_sum<TPR>(q.x + q.y, xch, turn) * inv_d + p.eps);
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
    const uint32_t xm = SHIFT ? row_shift(static_cast<const uint8_t*>(p.x) + row * p.ldx * ES) : 0;
    const uint32_t rm = SHIFT ? row_shift(static_cast<const uint8_t*>(p.resid) + row * p.ldr * ES) : 0;
    uint64_t v[NV][PP];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (SHIFT) read_shifted<ELEM>(slot + j * WB, xm, (t + TPR * j) * EPC, p.D, v[j]);
      else unpack_word<ELEM>(lds16(slot + j * WB), v[j]);
    }
    uint32_t draws[NV][PP];  // drawn ahead of the sums, beside whose exchanges they cost least
    if (p.drop.cut) {
#pragma unroll
      for (int j = 0; j < NV; ++j) word_draws<EPC, SHIFT>(key, (t + TPR * j) * EPC, p.D, (uint32_t)row, draws[j]);
    }
    uint64_t rs2 = pk(1.f, 1.f);
    if (p.g1) {
      float mu;
      const float rs = stats(v, mu);
      rs2 = pk(rs, rs);
      if (t == 0 && active) {
        p.rs1[row] = rs;
        if (FULL && p.layer) p.mu1[row] = mu;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t f[PP];
      factors(0, j, f);
      if constexpr (FULL) {
        uint64_t b[PP];
        factors(2, j, b);
#pragma unroll
        for (int k = 0; k < PP; ++k) v[j][k] = fma_2(mul_2(v[j][k], rs2), f[k], b[k]);
      } else {
#pragma unroll
        for (int k = 0; k < PP; ++k) v[j][k] = mul_2(mul_2(v[j][k], rs2), f[k]);
      }
    }
    if (p.drop.cut) {  // (branches around whole rows: inside the words' loops they would keep their loads and sums apart)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int k = 0; k < PP; ++k) v[j][k] = drop_pair(v[j][k], draws[j][k], key.cutw);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t r[PP];
      if constexpr (SHIFT) {
#pragma unroll
        for (int k = 0; k < PP; ++k) r[k] = 0;
        if (p.resid) read_shifted<ELEM>(slot + TB + j * WB, rm, (t + TPR * j) * EPC, p.D, r);
      } else {
        unpack_word<ELEM>(lds16(slot + TB + j * WB), r);
      }
#pragma unroll
      for (int k = 0; k < PP; ++k) v[j][k] = fma_2(v[j][k], scale2, r[k]);  // zeros past D
      const uint4 u = pack_word<ELEM>(v[j]);
      unpack_word<ELEM>(u, v[j]);  // normalised as it is kept
      if constexpr (SHIFT) write_shifted<ELEM, TPR>(hp - t * 16, (t + TPR * j) * EPC, p.D, t, active, u);
      else if (active && (t + TPR * j) * EPC < p.D) *reinterpret_cast<uint4*>(hp + TPR * j * 16) = u;
    }
    last = slot;
    slot = slot == mine + P * SB ? mine : slot + SB;
    hp += p.hstep;
    if (!p.g2) continue;
    float mu;
    const float rs = stats(v, mu);
    if (SHIFT || active) {
      rs2 = pk(rs, rs);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!SHIFT && (t + TPR * j) * EPC >= p.D) continue;
        uint64_t f[PP];
        factors(1, j, f);
        if constexpr (FULL) {
          uint64_t b[PP];
          factors(3, j, b);
#pragma unroll
          for (int k = 0; k < PP; ++k) v[j][k] = fma_2(mul_2(v[j][k], rs2), f[k], b[k]);
        } else {
#pragma unroll
          for (int k = 0; k < PP; ++k) v[j][k] = mul_2(mul_2(v[j][k], rs2), f[k]);
        }
        if constexpr (SHIFT) write_shifted<ELEM, TPR>(yp - t * 16, (t + TPR * j) * EPC, p.D, t, active, pack_word<ELEM>(v[j]));
        else *reinterpret_cast<uint4*>(yp + TPR * j * 16) = pack_word<ELEM>(v[j]);
      }
      if (t == 0 && active) {
        p.rs2[row] = rs;
        if (FULL && p.layer) p.mu2[row] = mu;
      }
    }
    yp += p.ystep;
  }
  cp_wait<0>();
}

// ------------------------------------------------------------ host side
template <int ELEM, int TPR, int NE>
lnfp8_status fwd_any_launch(const JoinFwdParams& p, cudaStream_t st) {
  constexpr auto kernel = join_fwd_any_kernel<ELEM, TPR, NE>;
  constexpr int threads = TPR < 256 ? 256 : TPR, gpb = threads / TPR;
  int bps = 1;
  const lnfp8_status s = kernel_setup<kernel>(threads, 0, &bps, "block_join_fwd: kernel set-up");
  if (s != LNFP8_OK) return s;
  // blocks that are all resident: each reads the columns' factors once
  const int64_t blocks = min64((p.M + gpb - 1) / gpb, (int64_t)num_sms() * bps);
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, p) != cudaSuccess) return check_launch("block_join_fwd launch");
  return check_launch("block_join_fwd");
}
template <int ELEM>
lnfp8_status fwd_any(const JoinFwdParams& p, cudaStream_t st) {
  if constexpr (ELEM == LNFP8_FP32) {
    if (p.D <= 256) return fwd_any_launch<ELEM, 32, 8>(p, st);
    if (p.D <= 512) return fwd_any_launch<ELEM, 64, 8>(p, st);
    if (p.D <= 1024) return fwd_any_launch<ELEM, 128, 8>(p, st);
    if (p.D <= 2048) return fwd_any_launch<ELEM, 256, 8>(p, st);
    if (p.D <= 4096) return fwd_any_launch<ELEM, 512, 8>(p, st);
    if (p.D <= 8192) return fwd_any_launch<ELEM, 1024, 8>(p, st);
  }
  return fwd_any_launch<ELEM, 1024, 16>(p, st);
}

template <int ELEM, int TPR, int NV, bool FULL, bool SHIFT = false>
lnfp8_status fwd_vec_launch(const JoinFwdParams& p, cudaStream_t st) {
  using S = JoinFwdShape<ELEM, TPR, NV, FULL, SHIFT>;
  constexpr auto kernel = join_fwd_vec_kernel<ELEM, TPR, NV, FULL, SHIFT>;
  const lnfp8_status s = kernel_setup<kernel>(kVecThreads, S::SMEM, nullptr, "block_join_fwd: kernel set-up");
  if (s != LNFP8_OK) return s;
  constexpr int gpb = kVecThreads / TPR, es = ElemSize<ELEM>::value;
  const int64_t blocks = min64(p.M, num_sms());
  JoinFwdParams q = p;
  q.step = blocks * gpb;
  q.xstep = q.step * p.ldx * es;
  q.rstep = q.step * p.ldr * es;
  q.hstep = q.step * p.ldh * es;
  q.ystep = q.step * p.ldy * es;
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(kVecThreads), S::SMEM, st, q) != cudaSuccess) return check_launch("block_join_fwd launch");
  return check_launch("block_join_fwd");
}
// Columns a thread: 16; 24 (16-bit types) where those would leave a quarter of the threads or more without any; 32 where a row is
// much work, whose exchanges then cost an SM less. Rows of one RMS norm without draws wait for memory alone and keep 16 from 2048
// columns on. us, bf16, 16 columns and the ones taken:
//                                           16384 x 1024  16384 x 2048  16384 x 2560  8192 x 4096  8192 x 5120  4096 x 8192
//   two layer norms, betas and a gate       31 and 27     56 and 47     108 and 72    64 and 50    120 and 80   71 (16)
//   one layer norm with betas, dropout      27 and 26     50 and 47     91 and 68     54 and 48    99 and 70    57 (16)
//   two RMS norms, dropout                  24 (16)       45 (16; 48)   84 and 60     48 (16; 47)  97 and 66    57 and 49
//   two RMS norms                           24 (16)       47 (16; 48)   65 and 62     46 (16; 49)  75 and 60    45 (16; 51)
//   one RMS norm                            23 (16)       46 (16; 47)   53 (16; 61)   47 (16; 47)  56 (16; 60)  47 (16; 48)
// (in brackets the columns taken, then the time of the others). One layer norm without draws keeps 16 too (2048 columns 44, 48).
template <int ELEM, bool FULL>
lnfp8_status fwd_vec16(const JoinFwdParams& p, cudaStream_t st) {
  const bool some = FULL || p.g1 || p.drop.cut, much = (p.g1 && p.drop.cut) || (FULL && (p.g1 || p.drop.cut));
  if (p.D <= 128) return fwd_vec_launch<ELEM, 8, 2, FULL>(p, st);
  if (p.D <= 256) return fwd_vec_launch<ELEM, 16, 2, FULL>(p, st);
  if (p.D <= 512) return fwd_vec_launch<ELEM, 32, 2, FULL>(p, st);
  if (p.D <= 32 * 24) return fwd_vec_launch<ELEM, 32, 3, FULL>(p, st);
  if constexpr (FULL)
    if (much && p.D <= 1024) return fwd_vec_launch<ELEM, 32, 4, FULL>(p, st);
  if (p.D <= 1024) return fwd_vec_launch<ELEM, 64, 2, FULL>(p, st);
  if (p.D <= 64 * 24) return fwd_vec_launch<ELEM, 64, 3, FULL>(p, st);
  if constexpr (FULL)
    if (much && p.D <= 2048) return fwd_vec_launch<ELEM, 64, 4, FULL>(p, st);
  if (p.D <= 2048) return fwd_vec_launch<ELEM, 128, 2, FULL>(p, st);
  if (some && p.D <= 128 * 24) return fwd_vec_launch<ELEM, 128, 3, FULL>(p, st);
  if constexpr (FULL)
    if (much && p.D <= 4096) return fwd_vec_launch<ELEM, 128, 4, FULL>(p, st);
  if (p.D <= 4096) return fwd_vec_launch<ELEM, 256, 2, FULL>(p, st);
  if (some && p.D <= 256 * 24) return fwd_vec_launch<ELEM, 256, 3, FULL>(p, st);
  if constexpr (!FULL)  // (four factors a column would not fit beside two rows)
    if (much && p.D <= 8192) return fwd_vec_launch<ELEM, 256, 4, FULL>(p, st);
  return p.D <= 8192 ? fwd_vec_launch<ELEM, 512, 2, FULL>(p, st) : fwd_vec_launch<ELEM, 512, 4, FULL>(p, st);
}
template <bool FULL>
lnfp8_status fwd_vec32(const JoinFwdParams& p, cudaStream_t st) {
  constexpr int E = LNFP8_FP32;
  if (p.D <= 128) return fwd_vec_launch<E, 8, 4, FULL>(p, st);
  if (p.D <= 256) return fwd_vec_launch<E, 16, 4, FULL>(p, st);
  if (p.D <= 512) return fwd_vec_launch<E, 32, 4, FULL>(p, st);
  if (p.D <= 1024) return fwd_vec_launch<E, 64, 4, FULL>(p, st);
  if (p.D <= 2048) return fwd_vec_launch<E, 128, 4, FULL>(p, st);
  return p.D <= 4096 ? fwd_vec_launch<E, 256, 4, FULL>(p, st) : fwd_any<E>(p, st);
}
template <int ELEM>
lnfp8_status fwd_shift(const JoinFwdParams& p, cudaStream_t st) {
  if (p.D <= 128) return fwd_vec_launch<ELEM, 8, 2, true, true>(p, st);
  if (p.D <= 256) return fwd_vec_launch<ELEM, 16, 2, true, true>(p, st);
  if (p.D <= 512) return fwd_vec_launch<ELEM, 32, 2, true, true>(p, st);
  if (p.D <= 1024) return fwd_vec_launch<ELEM, 64, 2, true, true>(p, st);
  if (p.D <= 2048) return fwd_vec_launch<ELEM, 128, 2, true, true>(p, st);
  if (p.D <= 4096) return fwd_vec_launch<ELEM, 256, 2, true, true>(p, st);
  return fwd_vec_launch<ELEM, 512, 2, true, true>(p, st);
}
// Rows on 16-byte boundaries (in fp32 up to 4096 columns) take the kernel of 16-byte words, others of a 16-bit type its form that
// shifts them, up to 8192 columns (8191 x 1001 fp16 with a gate and two layer norms 44 us by single elements, 30 shifted; fp32,
// whose elements are half the accesses a byte, 100000 x 203 67 and 96). All else goes by single elements.
template <int ELEM>
lnfp8_status fwd(const JoinFwdParams& p, cudaStream_t st) {
  constexpr int es = ElemSize<ELEM>::value;
  const bool vec = p.D % 8 == 0 && row_aligned(p.x, p.ldx, es) && row_aligned(p.h, p.ldh, es) &&
                   (!p.resid || row_aligned(p.resid, p.ldr, es)) && (!p.g2 || row_aligned(p.y, p.ldy, es)) &&
                   (p.D <= 8192 || vectors_aligned({p.g1, p.b1, p.gate, p.g2, p.b2}));
  if (!vec) {
    if constexpr (ELEM != LNFP8_FP32)
      if (p.D <= 8192) return fwd_shift<ELEM>(p, st);
    return fwd_any<ELEM>(p, st);
  }
  const bool full = (p.layer && (p.g1 || p.g2)) || p.b1 || p.b2;
  if constexpr (ELEM == LNFP8_FP32) return full ? fwd_vec32<true>(p, st) : fwd_vec32<false>(p, st);
  else return full ? fwd_vec16<ELEM, true>(p, st) : fwd_vec16<ELEM, false>(p, st);
}

}  // namespace

lnfp8_status block_join_fwd_launch(const lnfp8_block_join_fwd_args* a, cudaStream_t st) {
  if (a->M == 0) return drop_save_launch(a->drop, "block_join_fwd", st);
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
  if (a->elem == LNFP8_BF16) return fwd<LNFP8_BF16>(p, st);
  return a->elem == LNFP8_FP16 ? fwd<LNFP8_FP16>(p, st) : fwd<LNFP8_FP32>(p, st);
}

}  // namespace lnfp8
