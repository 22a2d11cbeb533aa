// Included by linear.cu: the persistent kernel.
//
// A pair of CTAs (a cluster of 2) computes 256 x BN tiles with the 2-SM MMA
// (256 x BN x 16 per instruction): each CTA loads its 128 rows of A and half of the
// B tile by TMA into its own ring and signals the leader's barrier; one lane of the leader
// issues the MMAs for both. Two accumulators (2 x BN tensor-memory columns)
// alternate, so that the epilogue of one tile runs under the MMAs of the next.
//   warp 0      TMA producer          warp 1   tensor memory, MMA issuer (leader)
//   warps 2-3   idle                  warps 4-19  epilogue, 8 per accumulator
// An epilogue warp takes 32 rows (its tensor-memory lanes) and half of the tile's
// columns, 32 x 32 at a time: a thread holds 32 columns of one row, which is one
// checkpoint block, so the scale needs no exchange between threads.

// A launch computes one product with the full epilogue (the forward), or up to two plain ones (the
// backward's dx and dw, independent of one another): their tiles are one list, so that the last
// round of the persistent loop is incomplete once, not twice (8192 x 2048 x 8192: 256 + 256 tiles on 76
// pairs are 7 rounds instead of 4 + 4).
enum LinEpi {
  LIN_FULL = 0,   // bias, saved pre-activation, activation, residual; both operands K-major
  LIN_PLAIN = 1,  // out = T(acc), or T(acc * cscale[col] + rvec[row] * cvec[col]); A either way, B MN-major
};

constexpr int kPairEpiWarps = 16;
constexpr int kPairThreads = 128 + 32 * kPairEpiWarps;

template <int BN>
struct PairCfg {
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = BN / 2 * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  // The ring takes all of shared memory but the bias slots: the way from a stage's release to its next data (barrier,
  // TMA, L2, the leader's barrier) is about 1500 cycles and a stage's MMAs 512 or fewer, so four stages leave the
  // tensor cores waiting: 16384 x 8192 x 2048 took 340 us with four and staged boxes, 312 with seven. The epilogue
  // has no staging: a thread's 32 columns are whole 32-byte sectors of its row, and are stored and loaded so.
  static constexpr int STAGES = (232448 - 1024 - 256 - 64 * kPairEpiWarps) / STAGE;
  static constexpr int BAR_OFF = STAGES * STAGE;
  static constexpr int BIAS_OFF = BAR_OFF + 256;  // a chunk's 32 columns of the bias for each epilogue warp
  static constexpr int SMEM = 1024 + BIAS_OFF + 64 * kPairEpiWarps;
  static constexpr int TMEM_COLS = 2 * BN;
  static_assert(STAGES >= 4 && SMEM <= 232448, "shared memory budget");
};

struct PairProb {
  int M, N, num_m2, num_n, num_kb, group_m, tiles, a_mn;
  int pieces, kb_per_piece;  // K pieces of a tile, neighbours in the list; `tiles` counts them
  uint32_t idesc;
  int wide_out;        // rows of out on 32-byte boundaries
  void* out;
  int64_t ldo;
  float* part;         // with pieces > 1: [pieces][M][N] fp32 instead, on a 32-byte boundary
  const void* cscale;  // with cvec and rvec, or NULL
  const void* cvec;
  const float* rvec;
};

struct PairParams {
  PairProb prob[2];
  int tiles;  // of both
  // the full epilogue
  int f16, act, ck, wide_resid, wide_h, wide_codes;
  const void* bias;
  const void* resid;
  int64_t ldr;
  void* h;
  uint8_t* codes;
  uint8_t* scales;
  int64_t pitch;
};

struct PairMaps {
  CUtensorMap a[2], b[2];
};

// Tile t of a [num_m2 x num_n] grid: M fastest inside groups of G, then N, then the next
// group; G panels of A stay in L2 while the group's columns pass.
__device__ __forceinline__ int2 pair_tile(int t, int num_m2, int num_n, int G) {
  const int span = G * num_n, grp = t / span, r = t - grp * span, m0 = grp * G;
  const int gs = min(G, num_m2 - m0);
  return make_int2(m0 + r % gs, r / gs);
}

// The product, tile and K blocks of position t in the list.
struct PairTile {
  int prob, m2, n, piece, kb0, kb1;
};
__device__ __forceinline__ PairTile pair_locate(const PairParams& p, int t) {
  const int q = t >= p.prob[0].tiles ? 1 : 0;
  const PairProb& r = p.prob[q];
  int u = q ? t - p.prob[0].tiles : t, piece = 0;
  if (r.pieces > 1) {
    piece = u % r.pieces;
    u /= r.pieces;
  }
  const int2 mn = pair_tile(u, r.num_m2, r.num_n, r.group_m);
  const int kb0 = piece * r.kb_per_piece;
  return {q, mn.x, mn.y, piece, kb0, min(r.num_kb, kb0 + r.kb_per_piece)};
}

// 32-byte accesses (sm_100 and later)
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
// 32 columns n0.. of a row of 16-bit elements: those below N (a multiple of 8).
__device__ __forceinline__ void store_row32(uint16_t* row, int n0, int N, int wide, const uint64_t* z, int f16) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 v = upk(z[i]);
    w[i] = pack16(v.x, v.y, f16);
  }
  if (wide && n0 + 32 <= N) {
    store32(row + n0, w);
    store32(row + n0 + 16, w + 8);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n0 + 8 * j < N) *reinterpret_cast<uint4*>(row + n0 + 8 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
}
__device__ __forceinline__ void load_row32(const uint16_t* row, int n0, int N, int wide, uint32_t* w) {
  if (wide && n0 + 32 <= N) {
    load32(row + n0, w);
    load32(row + n0 + 16, w + 8);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 u = n0 + 8 * j < N ? *reinterpret_cast<const uint4*>(row + n0 + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
      w[4 * j] = u.x;
      w[4 * j + 1] = u.y;
      w[4 * j + 2] = u.z;
      w[4 * j + 3] = u.w;
    }
  }
}

// A pair's unit of round r: the rounds run forwards and backwards in turn, so that the pairs that got
// the longer units of a round (they come first) get the later ones of the next.
__device__ __forceinline__ int pair_unit(int r, int cid, int ncl) { return r * ncl + (r & 1 ? ncl - 1 - cid : cid); }

// The activation of 32 values held as 16 pairs.
template <int ACT>
__device__ __forceinline__ void act_pairs(uint64_t* z) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) act8<ACT>(z + i);
}

template <int BN, int EPI>
__global__ void __launch_bounds__(kPairThreads, 1)
lin_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p) {
  using C = PairCfg<BN>;
  constexpr bool B_MN = EPI == LIN_PLAIN;
  static_assert(!B_MN || BN >= 128, "a CTA's half of an MN-major tile is whole boxes of 64 columns");
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  const uint32_t bar0 = ring + C::BAR_OFF;
  // full[STAGES], empty[STAGES], tfull[2], tempty[2], drain
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
  static_assert(8 * (2 * STAGES + 5) + 8 <= 256, "barrier space");
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::BAR_OFF + 8 * (2 * STAGES + 5));
  volatile uint32_t* abort_flag = misc;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kPairEpiWarps);  // the 8 warps of this buffer in both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_map(&maps.a[0]);
    tma_prefetch_map(&maps.b[0]);
  }
  cluster_sync_all();  // the peer signals this CTA's barriers
  if (warp == 1) tmem_alloc<true>(smem_u32((const void*)(misc + 1)), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, misc[1], 0);
  pdl_wait();
  pdl_launch_dependents();

  const int rank = blockIdx.x & 1;  // in the cluster
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  const int tiles = p.tiles;

  if (warp == 0) {
    // (this loop and the MMA issuer's share their schedulers with busy epilogue warps: a K block's instructions are
    // the pipeline's slowest part unless they are few, so addresses and descriptors only move by additions)
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    const uint32_t fb0 = map_to_rank(full_bar(0), 0);
    for (int rd = 0; ok; ++rd) {
      const int t = pair_unit(rd, cid, ncl);
      if (t >= tiles) break;
      const PairTile at = pair_locate(p, t);
      const CUtensorMap *tmA = &maps.a[at.prob], *tmB = &maps.b[at.prob];
      const bool a_mn = EPI == LIN_PLAIN && p.prob[at.prob].a_mn;
      const int m0 = at.m2 * 256 + rank * 128, n0 = at.n * BN + rank * (BN / 2);
      for (int kb = at.kb0; kb < at.kb1; ++kb) {
        if (!mbar_wait_warp(empty_bar(stage), phase ^ 1, abort_flag)) { ok = false; break; }
        if (one) {
          const uint32_t fb = fb0 + 8u * stage;
          const uint32_t ad = ring + stage * C::STAGE, bd = ad + C::A_BYTES;
          if (rank == 0) mbar_expect_tx(full_bar(stage), 2 * C::STAGE);
          if (!a_mn) tma_load_pair(ad, tmA, kb * BK, m0, fb);
          else {
            tma_load_pair(ad, tmA, m0, kb * BK, fb);
            tma_load_pair(ad + 8192, tmA, m0 + 64, kb * BK, fb);
          }
          if constexpr (!B_MN) tma_load_pair(bd, tmB, kb * BK, n0, fb);
          else
#pragma unroll
            for (int j = 0; j < BN / 128; ++j) tma_load_pair(bd + j * 8192, tmB, n0 + 64 * j, kb * BK, fb);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
    }
    // the commits behind the last stages signal both CTAs' barriers, which stay until every signal has come (a stage
    // that was never filled counts as released)
    for (int i = 0, s = stage, ph = phase; ok && i < STAGES; ++i) {
      ok = mbar_wait_warp(empty_bar(s), ph ^ 1, abort_flag);
      if (++s == STAGES) { s = 0; ph ^= 1; }
    }
    if (!ok && rank == 0 && one)
      for (int64_t i = min64(issued, STAGES); i > 0; --i) {
        if (--stage < 0) { stage = STAGES - 1; phase ^= 1; }
        mbar_drain(full_bar(stage), phase);
      }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const bool one = elect_one();
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const MatDesc bdesc = mat_desc(ring + C::A_BYTES, B_MN);
      for (int rd = 0; ok; ++rd) {
        const int t = pair_unit(rd, cid, ncl);
        if (t >= tiles) break;
        if (!mbar_wait_warp(tempty_bar(acc), acc_phase ^ 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const PairTile at = pair_locate(p, t);
        const PairProb& pr = p.prob[at.prob];
        const uint32_t idesc = pr.idesc;
        const MatDesc adesc = mat_desc(ring, EPI == LIN_PLAIN && pr.a_mn);
        const uint32_t d = tmem + (uint32_t)(acc * BN);
        for (int kb = at.kb0; kb < at.kb1; ++kb) {
          if (!mbar_wait_warp(full_bar(stage), phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          if (one) {
            const uint32_t off = stage * (C::STAGE >> 4);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_16bit<true>(d, mat_desc64(adesc.lo + off + kk * adesc.k_step), mat_desc64(bdesc.lo + off + kk * bdesc.k_step), idesc,
                              kk != 0 || kb != at.kb0);
            mma_commit<true>(empty_bar(stage));
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (one) mma_commit<true>(tfull_bar(acc));
        __syncwarp();
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok && one) {  // no MMA may still write tensor memory when it is freed
        mma_commit<true>(drain_bar, 1);
        mbar_drain(drain_bar, 0);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    const int ew = warp - 4, acc = ew >> 3, quarter = warp & 3, half = (ew >> 2) & 1;
    constexpr int HALF = BN / 2, CHUNKS = HALF / 32;
    uint32_t acc_phase = 0;
    const uint32_t tempty = map_to_rank(tempty_bar(acc), 0), bias_slot = ring + C::BIAS_OFF + 64 * ew;
    // this group's rounds have its parity: a step of two rounds keeps the direction
    const int t0 = pair_unit(acc, cid, ncl);
    for (int t = t0; t < tiles; t += 2 * ncl) {
      const PairTile at = pair_locate(p, t);
      const PairProb& pr = p.prob[at.prob];
      const int m = at.m2 * 256 + rank * 128 + quarter * 32 + lane;
      const int nh = at.n * BN + half * HALF;  // this warp's first column
      const bool affine = EPI == LIN_PLAIN && pr.cscale != nullptr && pr.pieces == 1;
      const float rv = affine && m < pr.M ? __ldg(pr.rvec + m) : 0.f;
      const bool biased = EPI == LIN_FULL && p.bias != nullptr;
      // two columns a lane (16 lanes), a chunk ahead
      auto bias_word = [&](int n) {
        return lane < 16 && n + 2 * lane < pr.N ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.bias) + n) + lane) : 0u;
      };
      uint32_t next_bias = biased ? bias_word(nh) : 0u;
      if (!mbar_wait_warp(tfull_bar(acc), acc_phase, abort_flag)) break;  // the whole warp: what follows is warp-wide
      tc_fence_after();
      const bool row_ok = m < pr.M;
      uint32_t scale_word = 0;
#pragma unroll 1
      for (int ch = 0; ch < CHUNKS; ++ch) {
        const int n0 = nh + ch * 32;
        __syncwarp();  // rows past M took other branches; the bias slot has been read
        if (biased) {
          if (lane < 16) sts4(bias_slot + 4 * lane, next_bias);
          if (ch + 1 < CHUNKS) next_bias = bias_word(n0 + 32);
          __syncwarp();
        }
        uint32_t rr[32];
        tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * BN + half * HALF + ch * 32), rr);
        if (ch == CHUNKS - 1 && t + 2 * ncl < tiles) {  // someone waits for it: nothing is in flight when the CTA leaves
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(tempty);
        }
        uint64_t z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = pk(__uint_as_float(rr[2 * i]), __uint_as_float(rr[2 * i + 1]));
        if (EPI == LIN_PLAIN && pr.pieces > 1) {  // the piece's sums
          if (row_ok) {
            float* dst = pr.part + ((int64_t)at.piece * pr.M + m) * pr.N + n0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (n0 + 8 * j < pr.N) store32(dst + 8 * j, rr + 8 * j);
          }
          continue;
        }
        uint32_t res[16];
        if constexpr (EPI == LIN_FULL)
          if (p.resid && row_ok) load_row32(reinterpret_cast<const uint16_t*>(p.resid) + m * p.ldr, n0, pr.N, p.wide_resid, res);
        // every lane needs the same 32 columns: broadcast from the warp's slot (16 shuffles instead: 8192 x 2048 x 8192
        // 158 -> 161 us; from global memory in place: 16384 x 768 x 768 17 -> 21 us, each chunk waiting for L2)
        if (biased) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 bu = lds16(bias_slot + 16 * j);
            const uint32_t bw[4] = {bu.x, bu.y, bu.z, bu.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 b = unpack16(bw[i], p.f16);
              z[4 * j + i] = add_2(z[4 * j + i], pk(b.x, b.y));
            }
          }
        }
        if (affine) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (n0 + 8 * j >= pr.N) break;
            const uint4 su = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pr.cscale) + n0 + 8 * j));
            const uint4 vu = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pr.cvec) + n0 + 8 * j));
            const uint32_t sw[4] = {su.x, su.y, su.z, su.w}, vw[4] = {vu.x, vu.y, vu.z, vu.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 c = unpack16(sw[i], p.f16), v = unpack16(vw[i], p.f16);
              z[4 * j + i] = fma_2(z[4 * j + i], pk(c.x, c.y), mul_2(pk(rv, rv), pk(v.x, v.y)));
            }
          }
        }
        if constexpr (EPI == LIN_FULL) {
          if (p.h && row_ok) store_row32(reinterpret_cast<uint16_t*>(p.h) + (int64_t)m * pr.N, n0, pr.N, p.wide_h, z, p.f16);
          if (p.ck >= 0) {
            // columns past N are zero (no operand, no bias) and do not move the block's maximum
            float am = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 v = upk(z[i]);
              am = amax3(am, v.x, v.y);
            }
            const uint32_t b = ckpt_byte(abs_bits(am), p.ck);
            const float inv = ckpt_inv_scale(b);
            const uint64_t i2 = pk(inv, inv);
            scale_word |= b << (8 * ch);
            uint32_t q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 u = upk(mul_2(z[2 * i], i2)), v = upk(mul_2(z[2 * i + 1], i2));
              q[i] = fp8x2(u.x, u.y, p.ck) | (fp8x2(v.x, v.y, p.ck) << 16);
            }
            if (row_ok) {
              uint8_t* dst = p.codes + (int64_t)m * pr.N + n0;
              if (p.wide_codes && n0 + 32 <= pr.N) {
                store32(dst, q);
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (n0 + 8 * j < pr.N) reinterpret_cast<uint2*>(dst)[j] = make_uint2(q[2 * j], q[2 * j + 1]);
              }
            }
          }
          if (p.act == LNFP8_ACT_GELU) act_pairs<LNFP8_ACT_GELU>(z);
          else if (p.act == LNFP8_ACT_SILU) act_pairs<LNFP8_ACT_SILU>(z);
          else if (p.act == LNFP8_ACT_RELU) act_pairs<LNFP8_ACT_RELU>(z);
          if (p.resid && row_ok) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 v = unpack16(res[i], p.f16);
              z[i] = add_2(z[i], pk(v.x, v.y));
            }
          }
        }
        if (row_ok) store_row32(reinterpret_cast<uint16_t*>(pr.out) + m * pr.ldo, n0, pr.N, pr.wide_out, z, p.f16);
      }
      if constexpr (EPI == LIN_FULL) {
        if (p.ck >= 0 && row_ok && nh < pr.N) {  // the four (or, at the edge, fewer) blocks' bytes, one word of the row
          uint8_t* sc = p.scales + (int64_t)m * p.pitch + (nh >> 5);
          if constexpr (CHUNKS == 4) *reinterpret_cast<uint32_t*>(sc) = scale_word;
          else if constexpr (CHUNKS == 2) *reinterpret_cast<uint16_t*>(sc) = (uint16_t)scale_word;
          else *sc = (uint8_t)scale_word;
        }
      }
      acc_phase ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_relaxed();  // both CTAs are done with the pair's tensor memory
  if (warp == 1) {
    tc_fence_after();
    tmem_free<true>(tmem, C::TMEM_COLS);
  }
  cluster_sync_relaxed();  // nobody leaves while the peer may still signal its barriers
}

// One product (EPI LIN_FULL), or one or two (LIN_PLAIN).
template <int BN, int EPI>
lnfp8_status pair_launch(const LinGemm* g, int count, cudaStream_t st) {
  using C = PairCfg<BN>;
  constexpr auto k = lin_pair_kernel<BN, EPI>;
  const lnfp8_status set = kernel_setup<k>(kPairThreads, C::SMEM, nullptr, "linear: kernel set-up");
  if (set != LNFP8_OK) return set;
  PairParams p = {};
  PairMaps maps;
  auto wide = [](const void* q, int64_t ld, int size) { return (int)(reinterpret_cast<uintptr_t>(q) % 32 == 0 && ld * size % 32 == 0); };
  bool ok = true;
  int64_t tiles = 0;
  // the product of more K blocks first: the short tiles fill the last round
  auto blocks = [](const LinGemm& q) { return q.K / (q.pieces > 1 ? q.pieces : 1); };
  const int first = count == 2 && blocks(g[1]) > blocks(g[0]) ? 1 : 0;
  for (int i = 0; i < count; ++i) {
    const LinGemm& q = g[i ^ first];
    PairProb& r = p.prob[i];
    r.M = (int)q.M;
    r.N = (int)q.N;
    r.num_m2 = (int)((q.M + 255) / 256);
    r.num_n = (int)((q.N + BN - 1) / BN);
    r.num_kb = (int)((q.K + BK - 1) / BK);
    // A panels (256 rows x K) of a raster group: what fits in 48 MB of L2
    r.group_m = (int)max64(1, min64((48ll << 20) / (512 * max64(q.K, 1)), r.num_m2));
    r.pieces = EPI == LIN_PLAIN && q.pieces > 1 ? q.pieces : 1;
    r.kb_per_piece = (r.num_kb + r.pieces - 1) / r.pieces;
    r.tiles = r.num_m2 * r.num_n * r.pieces;
    r.a_mn = q.a_mn;
    r.idesc = make_idesc(q.elem, 256, BN, q.a_mn, q.b_mn);
    r.cscale = q.cscale;
    r.cvec = q.cvec;
    r.rvec = q.rvec;
    tiles += (int64_t)r.num_m2 * r.num_n * r.pieces;
    r.out = q.out;
    r.ldo = q.ldo;
    r.part = q.part;
    r.wide_out = wide(q.out, q.ldo, 2);
    ok = ok && operand_map(&maps.a[i], q.a, q.a_mn, q.M, q.K, q.lda, 128) && operand_map(&maps.b[i], q.b, q.b_mn, q.N, q.K, q.ldb, BN / 2);
  }
  if (tiles > 0x3FFFFFFF) return set_error(LNFP8_ERR_UNSUPPORTED_SHAPE, "linear: too many tiles");
  p.tiles = (int)tiles;
  if (count == 1) {
    p.prob[1] = p.prob[0];
    maps.a[1] = maps.a[0];
    maps.b[1] = maps.b[0];
  }
  p.f16 = g->elem == LNFP8_FP16;
  p.ck = -1;
  if constexpr (EPI == LIN_FULL) {
    p.act = g->act;
    p.ck = g->ckpt.codes ? g->ckpt.dtype : -1;
    p.resid = g->resid;
    p.ldr = g->ldr;
    p.wide_resid = wide(g->resid, g->ldr, 2);
    p.h = g->h;
    p.wide_h = wide(g->h, g->N, 2);
    p.bias = g->bias;
    p.codes = g->ckpt.codes;
    p.scales = g->ckpt.scales;
    p.wide_codes = wide(g->ckpt.codes, g->N, 1);
    p.pitch = lnfp8_act_ckpt_scale_pitch(g->N);
  }
  if (!ok) return set_error(LNFP8_ERR_CUDA, "linear: cuTensorMapEncodeTiled failed (driver entry point or arguments)");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * max64(1, min64(tiles, num_sms() / 2))));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  LaunchScope ls("linear_pair", st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, maps, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(LNFP8_ERR_CUDA, "linear launch: %s", cudaGetErrorString(e));
  }
  return check_launch("linear");
}

// out = T(sum of the pieces, in order), with the affine epilogue: 8 columns a thread.
struct JoinParams {
  const float* part;
  int pieces, f16;
  int64_t M, N, ldo;
  void* out;
  const void* cscale;
  const void* cvec;
  const float* rvec;
};
__global__ void __launch_bounds__(256) lin_join_kernel(const JoinParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t n8 = p.N >> 3, total = p.M * n8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / n8;
    const int n = (int)(i - m * n8) * 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll 4
    for (int q = 0; q < p.pieces; ++q) {
      const float4* src = reinterpret_cast<const float4*>(p.part + ((int64_t)q * p.M + m) * p.N + n);
      const float4 a = __ldcs(src), b = __ldcs(src + 1);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    if (p.cscale) {
      float cs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, cv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      add16x8(cs, *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.cscale) + n), p.f16);
      add16x8(cv, *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.cvec) + n), p.f16);
      const float rv = p.rvec[m];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(v[k], cs[k], rv * cv[k]);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + m * p.ldo + n) = pack16x8(v, p.f16);
  }
}

lnfp8_status join_launch(const LinGemm& g, cudaStream_t st) {
  JoinParams p;
  p.part = g.part;
  p.pieces = g.pieces;
  p.f16 = g.elem == LNFP8_FP16;
  p.M = g.M;
  p.N = g.N;
  p.ldo = g.ldo;
  p.out = g.out;
  p.cscale = g.cscale;
  p.cvec = g.cvec;
  p.rvec = g.rvec;
  const int64_t blocks = min64((g.M * g.N / 8 + 255) / 256, (int64_t)num_sms() * 8);
  LaunchScope ls("linear_join", st);
  if (launch_pdl(lin_join_kernel, dim3((unsigned)blocks), dim3(256), 0, st, p) != cudaSuccess) return check_launch("linear_act_bwd launch");
  return check_launch("linear_act_bwd: joining K pieces");
}
