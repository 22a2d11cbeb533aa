// The 16-bit linear layer with bias, activation and residual in its epilogue, and
// its backward (te.Linear outside fp8_autocast, TE tutorial, code blocks 1 and 2:
// projections and head in 16 bits beside the FP8 modules):
//   forward   z = x w^T + b, y = T(act(z) + r); z kept as T(z) or as an 8-bit checkpoint
//   backward  dz = dy act'(h), db = sum_rows dz, dx = T(dz w), dw = T(dz^T x)
// The products run on the tensor cores (tcgen05, 16-bit operands staged by TMA,
// fp32 accumulators in tensor memory); the backward reads dz, w and x in the
// layouts they have (operands may be K-major or MN-major), so nothing is transposed.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "cp_async.cuh"
#include "internal.h"
#include "kernel_setup.cuh"
#include "rowmath.cuh"
#include "tc.cuh"

namespace lnfp8 {

lnfp8_status lin_status_read_clear(unsigned int* word) {
  const unsigned int zero = 0;
  if (cudaMemcpyFromSymbol(word, g_tc_status, sizeof(unsigned int)) != cudaSuccess ||
      (*word && cudaMemcpyToSymbol(g_tc_status, &zero, sizeof(unsigned int)) != cudaSuccess))
    return check_launch("lnfp8_sync_status: the linear layer's status word");
  return LNFP8_OK;
}

namespace {

constexpr int BK = 64;  // 16-bit elements of K per pipeline stage: 128-byte rows

struct EpiParams {
  int M, N, f16, act, ck;  // ck: -1 none, else the checkpoint's lnfp8_dtype
  void* out;
  int64_t ldo;
  const void* bias;
  const void* resid;
  int64_t ldr;
  void* h;
  uint8_t* codes;
  uint8_t* scales;
  int64_t pitch;
};

__device__ __forceinline__ uint32_t pack16(float a, float b, int f16) {
  if (f16) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ float2 unpack16(uint32_t w, int f16) {
  if (f16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack16x8(const float* v, int f16) {
  return make_uint4(pack16(v[0], v[1], f16), pack16(v[2], v[3], f16), pack16(v[4], v[5], f16), pack16(v[6], v[7], f16));
}
__device__ __forceinline__ void add16x8(float* v, uint4 u, int f16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack16(w[i], f16);
    v[2 * i] += p.x;
    v[2 * i + 1] += p.y;
  }
}

// The epilogue of 8 columns n.. of row m. The four lanes of a checkpoint block (32 columns)
// are neighbours; every lane of the warp calls it (`ok`: inside the tensor).
__device__ __forceinline__ void epilogue8(const EpiParams& p, float* v, int m, int n, bool ok) {
  const int64_t row = m;
  if (p.bias && ok) add16x8(v, *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.bias) + n), p.f16);
  if (p.h && ok)
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.h) + row * p.N + n) = pack16x8(v, p.f16);
  if (p.ck >= 0) {
    // items outside the tensor hold zeros
    const uint32_t b = ckpt_byte(block_amax8(v), p.ck);
    if (ok) {
      *reinterpret_cast<uint2*>(p.codes + row * p.N + n) = encode8(v, ckpt_inv_scale(b), p.ck);
      if ((n & 31) == 0) p.scales[row * p.pitch + (n >> 5)] = (uint8_t)b;
    }
  }
  if (p.act != LNFP8_ACT_NONE)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_fwd(v[i], p.act);
  if (ok) {
    if (p.resid) add16x8(v, *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.resid) + row * p.ldr + n), p.f16);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + row * p.ldo + n) = pack16x8(v, p.f16);
  }
}

// ------------------------------------------------------------ one tile per cluster
// A cluster computes one tile, its K cut into S pieces on S SMs (PAIR: S CTA pairs). The pieces'
// fp32 sums are then read from one another's shared memory and added in the pieces' order, each CTA
// finishing 1/S of its rows of the tile: no workspace, and the result does not depend on timing.
//   PAIR    the 2-SM MMA, 256 x BN x 16: a CTA holds 128 rows and loads half of the BN side. A
//           128 x 128 tile on one SM reads and fills 256 bytes of shared memory a clock, twice what
//           there is; a pair holds half of the BN side each (measured on 181 x 6392 x 7112: 52 -> 30 us). Taken
//           where K is long and the tiles are few: 256 x 4096 x 4096 13.9 us, 14.8 on persistent pairs.
//   SWAP    (up to 64 tokens) the accumulator's lanes are output features and its BN columns tokens, so that few
//           tokens fill the instruction; else lanes are tokens. 8 x 4096 x 4096 9.4 us, 3.6 TB/s.
template <int BN, bool PAIR>
struct TileCfg {
  static constexpr int P_BYTES = 128 * BK * 2;
  static constexpr int Q_BYTES = (PAIR ? BN / 2 : BN) * BK * 2;
  static constexpr int STAGE = P_BYTES + Q_BYTES;
  static constexpr int STAGES = 196608 / STAGE > 8 ? 8 : 196608 / STAGE;
  static constexpr int SMEM = 1024 + STAGES * STAGE + 256;
  static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(128 * (BN + 4) * 4 <= STAGES * STAGE, "the fp32 tile reuses the ring");
};

struct TileParams {
  EpiParams e;
  int num_p, num_kb, kb_per_split, p_mn, splits;
  uint32_t idesc;
};
struct TileMaps {
  CUtensorMap p, q;
};

constexpr int kTileThreads = 256;

template <int BN, bool PAIR, bool SWAP>
__global__ void __launch_bounds__(kTileThreads, 1)
lin_tile_kernel(const __grid_constant__ TileMaps maps, const __grid_constant__ TileParams p) {
  using C = TileCfg<BN, PAIR>;
  constexpr int STAGES = C::STAGES, SIDES = PAIR ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  const uint32_t bars = ring + STAGES * C::STAGE;  // full[STAGES], empty[STAGES], done
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + STAGES * C::STAGE + 8 * (2 * STAGES + 1));
  volatile uint32_t* abort_flag = misc;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (STAGES + s); };
  const uint32_t done_bar = bars + 8u * (2 * STAGES);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int S = p.splits;
  const bool clustered = S * SIDES > 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_map(&maps.p);
    tma_prefetch_map(&maps.q);
  }
  if constexpr (PAIR) cluster_sync_all();  // the peer signals this CTA's barriers
  if (warp == 1) tmem_alloc<PAIR>(smem_u32((const void*)(misc + 1)), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, misc[1], 0);
  pdl_wait();
  pdl_launch_dependents();

  const int crank = blockIdx.x % (S * SIDES);  // in the cluster
  const int side = PAIR ? crank & 1 : 0, piece = crank / SIDES, leader = crank - side;
  const CUtensorMap *tmP = &maps.p, *tmQ = &maps.q;
  const int tile = blockIdx.x / (S * SIDES);
  const int p0 = (tile % p.num_p) * (128 * SIDES) + side * 128, q0 = (tile / p.num_p) * BN;
  const int kb0 = piece * p.kb_per_split, kb1 = min(p.num_kb, kb0 + p.kb_per_split);
  const bool p_mn = p.p_mn != 0;
  const uint16_t both = (uint16_t)(3u << leader);

  if (warp == 0) {
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    bool ok = true;
    auto load = [&](uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
      if constexpr (PAIR) tma_load_pair(dst, tm, x, y, bar);
      else tma_load(dst, tm, x, y, bar);
    };
    const int qs = q0 + side * (BN / 2);  // the rows of Q this CTA loads
    const uint32_t fb0 = PAIR ? map_to_rank(full_bar(0), leader) : full_bar(0);
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(empty_bar(stage), phase ^ 1, abort_flag)) { ok = false; break; }
      if (one) {
        const uint32_t pd = ring + stage * C::STAGE, qd = pd + C::P_BYTES;
        const uint32_t fb = fb0 + 8u * stage;
        if (side == 0) mbar_expect_tx(full_bar(stage), SIDES * C::STAGE);
        if (!p_mn) load(pd, tmP, kb * BK, p0, fb);
        else {
          load(pd, tmP, p0, kb * BK, fb);
          load(pd + 8192, tmP, p0 + 64, kb * BK, fb);
        }
        load(qd, tmQ, kb * BK, qs, fb);
      }
      __syncwarp();
      ++issued;
      if (++stage == STAGES) { stage = 0; phase ^= 1; }
    }
    // the commits behind the last stages signal these barriers (PAIR: both CTAs'), which stay until every signal has come
    for (int i = 0, s = stage, ph = phase; ok && i < STAGES; ++i) {
      ok = mbar_wait_warp(empty_bar(s), ph ^ 1, abort_flag);
      if (++s == STAGES) { s = 0; ph ^= 1; }
    }
    if (!ok && side == 0 && one)
      for (int i = min(issued, STAGES); i > 0; --i) {  // copies in flight land before the CTA leaves
        if (--stage < 0) { stage = STAGES - 1; phase ^= 1; }
        mbar_drain(full_bar(stage), phase);
      }
    __syncwarp();
  } else if (warp == 1 && side == 0) {
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    const MatDesc pdesc = mat_desc(ring, p_mn), qdesc = mat_desc(ring + C::P_BYTES, false);
    const uint32_t idesc = p.idesc;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(full_bar(stage), phase, abort_flag)) break;
      tc_fence_after();
      if (one) {
        const uint32_t off = stage * (C::STAGE >> 4);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_16bit<PAIR>(tmem, mat_desc64(pdesc.lo + off + kk * pdesc.k_step), mat_desc64(qdesc.lo + off + kk * qdesc.k_step), idesc,
                          kk != 0 || kb != kb0);
        mma_commit<PAIR>(empty_bar(stage), both);
      }
      __syncwarp();
      if (++stage == STAGES) { stage = 0; phase ^= 1; }
    }
    if (one) mma_commit<PAIR>(done_bar, both);  // after an abort too: no MMA outlives the CTA
    __syncwarp();
  }

  // the fp32 tile, tokens by features, over the ring (every copy and MMA has completed)
  constexpr int ROWS = SWAP ? BN : 128, COLS = SWAP ? 128 : BN, PITCH = COLS + 4;
  float* tile_f = reinterpret_cast<float*>(smem);
  {
    uint32_t never = 0;
    mbar_wait(done_bar, 0, &never);
    __syncwarp();
    tc_fence_after();
    const int quarter = warp & 3;  // a warp's lanes of tensor memory; the two warps of a quarter take every other chunk
    const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
    for (int c = (warp >> 2) * 16; c < BN; c += 32) {
      uint32_t r[16];
      if (kb1 > kb0) tmem_ld16(t0 + c, r);
      else
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = 0u;
      if constexpr (SWAP) {
#pragma unroll
        for (int i = 0; i < 16; ++i) tile_f[(c + i) * PITCH + quarter * 32 + lane] = __uint_as_float(r[i]);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(tile_f + (quarter * 32 + lane) * PITCH + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (S > 1) cluster_sync_all();

  const int rows = ROWS / S;  // of this CTA; a multiple of 32 items in all
  constexpr int CH = COLS / 8;
  constexpr int kMostPieces = PAIR ? 2 : 4, U = PAIR ? 2 : 1;  // U items of a thread together
  for (int i0 = threadIdx.x; i0 < rows * CH; i0 += U * kTileThreads) {
    // every piece's words first: loads from another SM's shared memory take most of a microsecond. Items outside the
    // tensor load nothing: each value read from another CTA goes into a store to y, so that the thread has waited
    // for it before it reaches the barrier behind which that CTA may leave
    float4 a[U][kMostPieces], b[U][kMostPieces];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kTileThreads, r = piece * rows + i / CH, c = (i % CH) * 8;
      ok[u] = (SWAP ? q0 : p0) + r < p.e.M && (SWAP ? p0 : q0) + c < p.e.N;
      if (i >= rows * CH) break;
      if (!ok[u]) {
#pragma unroll
        for (int s = 0; s < kMostPieces; ++s) a[u][s] = b[u][s] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else if (S > 1) {
        const uint32_t at = ring + (uint32_t)(r * PITCH + c) * 4u;
#pragma unroll
        for (int s = 0; s < kMostPieces; ++s) {
          if (s >= S) break;
          const uint32_t ra = map_to_rank(at, s * SIDES + side);
          a[u][s] = ld_cluster_f4(ra);
          b[u][s] = ld_cluster_f4(ra + 16);
        }
      } else {
        a[u][0] = *reinterpret_cast<const float4*>(tile_f + r * PITCH + c);
        b[u][0] = *reinterpret_cast<const float4*>(tile_f + r * PITCH + c + 4);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kTileThreads, r = piece * rows + i / CH, c = (i % CH) * 8;
      if (i >= rows * CH) break;  // uniform over the warp
      float v[8] = {a[u][0].x, a[u][0].y, a[u][0].z, a[u][0].w, b[u][0].x, b[u][0].y, b[u][0].z, b[u][0].w};
#pragma unroll
      for (int s = 1; s < kMostPieces; ++s) {
        if (s >= S) break;
        v[0] += a[u][s].x; v[1] += a[u][s].y; v[2] += a[u][s].z; v[3] += a[u][s].w;
        v[4] += b[u][s].x; v[5] += b[u][s].y; v[6] += b[u][s].z; v[7] += b[u][s].w;
      }
      epilogue8(p.e, v, (SWAP ? q0 : p0) + r, (SWAP ? p0 : q0) + c, ok[u]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (clustered) cluster_sync_relaxed();  // nobody leaves while its tile may be read, nor frees the pair's tensor memory
  if (warp == 1) {
    tc_fence_after();
    tmem_free<PAIR>(tmem, C::TMEM_COLS);
  }
  if constexpr (PAIR) cluster_sync_relaxed();
}

// ------------------------------------------------------------ a few tokens
// One to four tokens (takes_few): bound by the weight's bytes, so each warp streams kRowsPerWarp rows of w with
// 16-byte loads straight into FMAs; x sits in shared memory in its own type. WK warps share a
// row group (K cut into WK pieces, added in order) when there are too few rows to fill the SMs.
// A lane's partial sum covers every 32nd group of 8 columns; a warp's lanes are added by shuffles.
constexpr int kRowsPerWarp = 2;
constexpr int kFewTokens = 4, kFewOutputs = 10240;
constexpr int kFewMaxX = 96 * 1024;  // bytes of x in shared memory

template <int MT, bool F16>
__global__ void __launch_bounds__(256) lin_few_kernel(const EpiParams e, const void* __restrict__ x, int64_t ldx,
                                                      const void* __restrict__ w, int K, int WK) {
  constexpr int ELEM = F16 ? LNFP8_FP16 : LNFP8_BF16;
  extern __shared__ uint4 xs[];  // [MT][K / 8]
  __shared__ float red[8][kRowsPerWarp][MT];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / WK, part = warp % WK;
  const int n0 = (blockIdx.x * (8 / WK) + group) * kRowsPerWarp;
  const int K8 = K >> 3;
  const int per = ((K8 + WK - 1) / WK + 31) / 32 * 32;  // 16-byte groups of a piece, whole warps of them
  const int k0 = part * per, k1 = min(K8, k0 + per);
  constexpr int U = 4;  // loads in flight per row
  uint4 wv[kRowsPerWarp][U];
  const uint4* wr[kRowsPerWarp];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) wr[r] = reinterpret_cast<const uint4*>(w) + (int64_t)min(n0 + r, e.N - 1) * K8;
  auto fetch = [&](int k) {
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k + 32 * u < k1) wv[r][u] = __ldcs(wr[r] + k + 32 * u);
  };
  fetch(k0 + lane);  // the first weights are on their way while x is staged
  for (int m = 0; m < MT; ++m)
    for (int k = threadIdx.x; k < K8; k += 256)
      xs[m * K8 + k] = m < e.M ? reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + m * ldx)[k] : make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  uint64_t acc[kRowsPerWarp][MT];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0;
  for (int k = k0 + lane; k < k1; k += 32 * U) {
    uint4 cur[kRowsPerWarp][U];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u) cur[r][u] = wv[r][u];
    fetch(k + 32 * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + 32 * u >= k1) break;
      uint64_t wf[kRowsPerWarp][4];
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) unpack8<ELEM>(&cur[r][u], wf[r]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint64_t xf[4];
        const uint4 xv = xs[m * K8 + k + 32 * u];
        unpack8<ELEM>(&xv, xf);
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][m] = fma_2(wf[r][i], xf[i], acc[r][m]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float2 t = upk(acc[r][m]);
      const float v = warp_sum(t.x + t.y);
      if (lane == 0) red[warp][r][m] = v;
    }
  __syncthreads();
  // one thread per (row group, row, token)
  const int i = threadIdx.x;
  if (i >= (8 / WK) * kRowsPerWarp * MT) return;
  const int m = i % MT, r = i / MT % kRowsPerWarp, g = i / (MT * kRowsPerWarp);
  const int n = (blockIdx.x * (8 / WK) + g) * kRowsPerWarp + r;
  if (m >= e.M || n >= e.N) return;
  float z = 0.f;
  for (int q = 0; q < WK; ++q) z += red[g * WK + q][r][m];
  if (e.bias) z += load_elem<ELEM>(e.bias, n);
  if (e.h) store_elem<ELEM>(e.h, (int64_t)m * e.N + n, z);
  z = act_fwd(z, e.act);
  if (e.resid) z += load_elem<ELEM>(e.resid, m * e.ldr + n);
  store_elem<ELEM>(e.out, m * e.ldo + n, z);
}

// ------------------------------------------------------------ dz = dy act'(h), db
// A block takes 256 columns (32 threads of 8) and `rows_per_block` rows, 8 at a time; each
// thread keeps the sums of its columns, added over the 8 row lanes at the end.
struct DactParams {
  const void* dy;
  const void* h;
  const uint8_t* codes;
  const uint8_t* scales;
  void* dz;      // NULL: no activation, only the column sums
  float* part;   // [row blocks][N] or NULL; with `both` [row blocks][2][N]: the sums of dz, then of dz as rounded
  int both;
  // or, from clusters of kDactCluster row blocks (dact_cluster_rows): the sums themselves
  float* db;
  float* dbr;
  int64_t M, lddy, pitch;
  int N, dt, rows_per_block;  // dt: the lnfp8_dtype of the codes
};

enum DactSource { DACT_NONE, DACT_TENSOR, DACT_CKPT };  // no activation; h as a tensor; h as a checkpoint
constexpr int kDactBlocksPerSm = 4;
constexpr int kDactCluster = 8;
// Up to how many rows the column sums come from clusters of 8 row blocks, without a second launch. Of the whole
// backward, us with one launch and with two, GELU from a checkpoint (tokens x K x N): 65 x 768 x 768 8.0 and 9.7, 256 x
// 4096 x 4096 32.3 and 33.0, 320 x 768 x 2304 19.3 and 18.8, 512 x 768 x 768 11.6 and 10.5, 1000 x 768 x 2304 32.1 and 19.8.
// Without an activation, where dy alone is read: 512 x 768 x 1536 10.0 and 10.9, 512 x 4096 x 4096 34.2 and 34.2, 1024 x 768
// x 1536 11.7 and 12.6, 1024 x 1024 x 1024 10.8 and 11.4, 1000 x 768 x 2304 17.5 and 15.4, 1024 x 1536 x 1536 18.6 and 16.8.
inline int64_t dact_cluster_rows(int64_t K, int64_t N, bool has_act) {
  return has_act ? 320 : K * N <= 3 << 19 ? 1024 : 512;
}

template <int SRC>
struct DactShape {
  static constexpr int H_OFF = 16, S_OFF = SRC == DACT_TENSOR ? 32 : 24;  // bytes per thread: dy, h or codes, scale word
  static constexpr int BYTES = SRC == DACT_NONE ? 16 : SRC == DACT_TENSOR ? 32 : 28;
  // Rows of a thread in its ring: all but one are on their way while that one is used. With h as a tensor six would leave
  // room for three blocks an SM, where the grid has four to one (8192 x 8192, GELU 94 us; six rows and a grid of three
  // 83; five rows 74, four 72; ReLU 65, 68, 67, 68; 8192 x 2048, GELU 28.4, 25.4, 23.8, 22.7, ReLU 20.3, 18.7, 19.0, 19.0).
  static constexpr int RING = SRC == DACT_TENSOR ? 4 : 6;
  static constexpr size_t SMEM = (size_t)RING * BYTES * 256;
  static constexpr size_t RED = 8 * 32 * 9 * sizeof(float);
  // of an SM's 228 KB each block takes 1 KB for itself
  static_assert(kDactBlocksPerSm * (SMEM + RED + 1024) <= 228 * 1024, "one wave of kDactBlocksPerSm blocks an SM");
};

template <int ELEM, int SRC, int ACT>
__global__ void __launch_bounds__(256, kDactBlocksPerSm) lin_dact_kernel(const DactParams p) {
  using S = DactShape<SRC>;
  constexpr int P = S::RING - 1;
  constexpr uint32_t SB = S::BYTES * 256;
  __shared__ float red[8][32][9];
  static_assert(sizeof(red) == S::RED);
  extern __shared__ uint4 ring[];  // [RING][BYTES * 256], each kind an array over the threads
  pdl_wait();
  pdl_launch_dependents();
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + cl) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * p.rows_per_block;
  const int64_t r1 = c < p.N ? min64(p.M, r0 + p.rows_per_block) : 0;
  uint64_t acc[4], accr[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = accr[k] = 0;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t a_dy = threadIdx.x * 16, a_h = S::H_OFF * 256 + threadIdx.x * (SRC == DACT_TENSOR ? 16 : 8),
                 a_s = S::S_OFF * 256 + threadIdx.x * 4;
  int64_t r = r0 + rl;
  const uint16_t* dyp = reinterpret_cast<const uint16_t*>(p.dy) + r * p.lddy + c;
  const uint16_t* hp = reinterpret_cast<const uint16_t*>(p.h) + r * p.N + c;
  const uint8_t* qp = p.codes + r * p.N + c;
  const uint8_t* sp = p.scales + r * p.pitch + ((c >> 7) << 2);  // the word that holds this column's scale byte
  const int64_t dystep = 8 * p.lddy, hstep = 8 * (int64_t)p.N, sstep = 8 * p.pitch;
  auto issue = [&](int64_t row, uint32_t slot) {
    if (row < r1) {
      cp16(slot + a_dy, dyp);
      dyp += dystep;
      if constexpr (SRC == DACT_TENSOR) {
        cp16(slot + a_h, hp);
        hp += hstep;
      } else if constexpr (SRC == DACT_CKPT) {
        cp8(slot + a_h, qp);
        cp4(slot + a_s, sp);
        qp += hstep;
        sp += sstep;
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int k = 0; k < P; ++k) issue(r + 8 * k, base + k * SB);
  uint32_t slot = base, last = base + P * SB;
  const int byte = ((c >> 5) & 3) * 8;
  uint16_t* zp = reinterpret_cast<uint16_t*>(p.dz) + r * p.N + c;
  for (; r < r1; r += 8) {
    issue(r + 8 * P, last);
    cp_wait<P>();
    uint64_t v[4];
    uint4 w = lds16(slot + a_dy);
    unpack8<ELEM>(&w, v);
    if constexpr (SRC != DACT_NONE) {
      uint64_t z[4], sl[4];
      uint32_t sb = 0;
      if constexpr (SRC == DACT_TENSOR) {
        w = lds16(slot + a_h);
        unpack8<ELEM>(&w, z);
      } else {
        sb = (lds4(slot + a_s) >> byte) & 0xFFu;
        decode8(lds8(slot + a_h), ckpt_scale(sb), p.dt, z);
      }
      // z^2 leaves fp32 only from bf16 values, or in blocks of scales above 2^40
      if (SRC == DACT_TENSOR ? ELEM == LNFP8_BF16 : sb >= 167u) slope8<ACT, true>(z, sl);
      else slope8<ACT, false>(z, sl);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = mul_2(v[k], sl[k]);
      pack8<ELEM>(v, &w);
      *reinterpret_cast<uint4*>(zp) = w;
      zp += hstep;
      if (p.both) {
        uint64_t u[4];
        unpack8<ELEM>(&w, u);
#pragma unroll
        for (int k = 0; k < 4; ++k) accr[k] = add_2(accr[k], u[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = add_2(acc[k], v[k]);
    last = slot;
    slot = slot == base + P * SB ? base : slot + SB;
  }
  cp_wait<0>();
  if (p.part == nullptr && p.db == nullptr) return;
  const int col = threadIdx.x;  // 256 columns
  float sum[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k > p.both) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = upk(k ? accr[i] : acc[i]);
      red[rl][cl][2 * i] = t.x;
      red[rl][cl][2 * i + 1] = t.y;
    }
    __syncthreads();
    sum[k] = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[k] += red[q][col >> 3][col & 7];
  }
  const int n = blockIdx.x * 256 + col;
  if (p.part != nullptr) {
    for (int k = 0; k <= p.both; ++k)
      if (n < p.N) p.part[((int64_t)blockIdx.y * (1 + p.both) + k) * p.N + n] = sum[k ? 1 : 0];
    return;
  }
  // the row blocks of a column block are one cluster: each adds an eighth of the columns over all of them
  __syncthreads();
  float* fin = &red[0][0][0];  // [2][256]
  fin[col] = sum[0];
  if (p.both) fin[256 + col] = sum[1];
  cluster_sync_all();
  const int rank = (int)cluster_rank(), lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  if (k <= p.both) {
    const uint32_t at = smem_u32(fin + 256 * k + rank * 32 + lane);
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < kDactCluster; ++q) t += ld_cluster_f(map_to_rank(at, q));
    const int m = blockIdx.x * 256 + rank * 32 + lane;
    if (m < p.N) (k ? p.dbr : p.db)[m] = t;
  }
  cluster_sync_all();  // nobody leaves while its sums may be read
}

// ------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// 2-D map over a row-major [outer, inner] tensor of 16-bit elements, row stride ld elements.
bool make_map(CUtensorMap* tm, const void* base, int64_t inner, int64_t outer, int64_t ld, int box_inner, int box_outer,
              CUtensorMapSwizzle swz) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)(ld * 2)};
  cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer};
  cuuint32_t estr[2] = {1u, 1u};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}
// An operand of `rows` rows/columns over K: `box_rows` of them per box when K-major, 64 when MN-major.
bool operand_map(CUtensorMap* tm, const void* base, bool mn, int64_t rows, int64_t K, int64_t ld, int box_rows) {
  return mn ? make_map(tm, base, rows, K, ld, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B)
            : make_map(tm, base, K, rows, ld, BK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// kind::f16: fp32 accumulator, both operands bf16 (1) or fp16 (0).
uint32_t make_idesc(int elem, int m_mma, int n_mma, bool a_mn, bool b_mn) {
  const uint32_t t = elem == LNFP8_BF16 ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n_mma >> 3) << 17) | ((uint32_t)(m_mma >> 4) << 24);
}

EpiParams epi_params(const LinGemm& g) {
  EpiParams e;
  e.M = (int)g.M;
  e.N = (int)g.N;
  e.f16 = g.elem == LNFP8_FP16;
  e.act = g.act;
  e.ck = g.ckpt.codes ? g.ckpt.dtype : -1;
  e.out = g.out;
  e.ldo = g.ldo;
  e.bias = g.bias;
  e.resid = g.resid;
  e.ldr = g.ldr;
  e.h = g.h;
  e.codes = g.ckpt.codes;
  e.scales = g.ckpt.scales;
  e.pitch = lnfp8_act_ckpt_scale_pitch(g.N);
  return e;
}

// S pieces of K per tile (1, 2 or 4; PAIR: 2). The lanes' operand (SWAP: b) may be MN-major, the other is K-major.
template <int BN, bool PAIR, bool SWAP>
lnfp8_status tile_launch(const LinGemm& q, int S, cudaStream_t st) {
  using C = TileCfg<BN, PAIR>;
  constexpr auto k = lin_tile_kernel<BN, PAIR, SWAP>;
  const lnfp8_status set = kernel_setup<k>(kTileThreads, C::SMEM, nullptr, "linear: kernel set-up");
  if (set != LNFP8_OK) return set;
  TileParams p = {};
  TileMaps maps;
  const int64_t prow = SWAP ? q.N : q.M, qrow = SWAP ? q.M : q.N;
  const bool p_mn = SWAP ? q.b_mn : q.a_mn;
  const int64_t num_p = (prow + (PAIR ? 255 : 127)) / (PAIR ? 256 : 128), num_q = (qrow + BN - 1) / BN, tiles = num_p * num_q;
  if (tiles > 0x0FFFFFFF) return set_error(LNFP8_ERR_UNSUPPORTED_SHAPE, "linear: too many tiles");
  p.e = epi_params(q);
  p.num_p = (int)num_p;
  p.num_kb = (int)((q.K + BK - 1) / BK);
  p.kb_per_split = (p.num_kb + S - 1) / S;
  p.splits = S;
  p.p_mn = p_mn;
  p.idesc = make_idesc(q.elem, PAIR ? 256 : 128, BN, p_mn, false);
  const bool ok = SWAP ? operand_map(&maps.p, q.b, p_mn, q.N, q.K, q.ldb, 128) && operand_map(&maps.q, q.a, false, q.M, q.K, q.lda, PAIR ? BN / 2 : BN)
                       : operand_map(&maps.p, q.a, p_mn, q.M, q.K, q.lda, 128) && operand_map(&maps.q, q.b, false, q.N, q.K, q.ldb, PAIR ? BN / 2 : BN);
  if (!ok) return set_error(LNFP8_ERR_CUDA, "linear: cuTensorMapEncodeTiled failed (driver entry point or arguments)");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S * (PAIR ? 2 : 1);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(tiles * S * (PAIR ? 2 : 1)));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  LaunchScope ls("linear_tile", st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, maps, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(LNFP8_ERR_CUDA, "linear launch: %s", cudaGetErrorString(e));
  }
  return check_launch("linear");
}

#include "linear_pair.cuh"

template <int ELEM, int SRC, int ACT>
lnfp8_status dact_launch(const DactParams& p, dim3 grid, cudaStream_t st) {
  constexpr auto k = lin_dact_kernel<ELEM, SRC, ACT>;
  const lnfp8_status set = kernel_setup<k>(256, DactShape<SRC>::SMEM, nullptr, "linear_act_bwd: kernel set-up");
  if (set != LNFP8_OK) return set;
  LaunchScope ls("linear_dact", st);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = kDactCluster;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = DactShape<SRC>::SMEM;
  cfg.stream = st;
  cfg.attrs = pdl_enabled() ? attr : attr + 1;
  cfg.numAttrs = (pdl_enabled() ? 1 : 0) + (p.db ? 1 : 0);
  if (cudaLaunchKernelEx(&cfg, k, p) != cudaSuccess) return check_launch("linear_act_bwd launch");
  return check_launch("linear_act_bwd: dz");
}

// Rows of the dz pass per block: one wave of resident blocks.
int64_t dact_rows_per_block(int64_t M, int64_t K, int64_t N, bool has_act) {
  if (M <= dact_cluster_rows(K, N, has_act)) return (M + 8 * kDactCluster - 1) / (8 * kDactCluster) * 8;
  const int64_t col_blocks = (N + 255) / 256;
  const int64_t row_blocks = max64(1, (int64_t)num_sms() * kDactBlocksPerSm / col_blocks);
  const int64_t rows = (M + row_blocks - 1) / row_blocks;
  return max64(32, (rows + 7) / 8 * 8);
}
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

namespace {
bool takes_swap(const LinGemm& g) { return g.M <= 64 && !g.a_mn; }

// How a product, or two in one launch, runs when lanes are tokens: the persistent kernel over tiles of 256, 128 or (K-major
// operands) 64 columns, or, forward, one 256 x 128 tile per cluster with K in two pieces. Costs in ns, fitted to
// measurements of all of them (36 shapes of 33 to 16384 tokens): a 64-wide K block takes a pair 270 (256 columns: the
// matrix rate) or 171 (128 and 64: the issue of copies and MMAs); the rest is launch, set-up, the last epilogue, and
// 500 a round. A tile takes no less than four K blocks' time, for its epilogue. Of the clusters of two pairs 36 fit on the
// chip at once. 333 x 768 x 2304 takes 5.8 us with 64 columns, 5.9 with 128, 8.2 with 256 and 8.3 with 128 in two
// pieces; 129 x 4096 x 4096 takes 14.6, 15.1, 22.7 and 13.8; 2048 x 2048 x 2048 takes 25.8, 16.4, 15.3 and 40.1.
struct LinPlan {
  int tile, S;  // S 1: the persistent kernel
};
// K blocks of the pair with the most: the list of units, longest first, dealt out forwards and backwards.
int64_t longest_pair(const int64_t* units, const int64_t* kb, int count, int64_t pairs) {
  const int first = count == 2 && kb[1] > kb[0] ? 1 : 0;
  const int64_t n0 = units[first], n = n0 + (count == 2 ? units[1 - first] : 0);
  const int64_t k0 = kb[first], k1 = count == 2 ? kb[1 - first] : 0;
  // rounds wholly of the first product cost every pair the same; look at what is left of them and the second
  int64_t worst = 0;
  for (int64_t c = 0; c < pairs; ++c) {
    int64_t sum = 0;
    const int64_t skip = n0 / (2 * pairs) * 2;
    sum += skip * k0;
    int64_t r = skip;
    for (; r * pairs < n && r < skip + 4; ++r) {
      const int64_t t = r * pairs + (r & 1 ? pairs - 1 - c : c);
      if (t < n) sum += t < n0 ? k0 : k1;
    }
    if (r * pairs < n) sum += ((n - r * pairs) + pairs - 1) / pairs * k1;
    worst = max64(worst, sum);
  }
  return worst;
}

LinPlan lin_plan(LinGemm* g, int count) {
  const int64_t pairs = max64(num_sms() / 2, 1);
  // the persistent kernel; pieces: a weight gradient's K in pieces
  auto persistent = [&](int bn, int64_t per_kb, int64_t fixed, bool pieces) {
    int64_t units[2] = {0, 0}, kb[2] = {0, 0}, join = 0;
    for (int i = 0; i < count; ++i) {
      const int64_t n = pieces && g[i].pieces > 1 ? g[i].pieces : 1;
      units[i] = (g[i].M + 255) / 256 * ((g[i].N + bn - 1) / bn) * n;
      kb[i] = max64(4, ((g[i].K + BK - 1) / BK + n - 1) / n);
      if (n > 1) join += 2000 + n * g[i].M * g[i].N * 8 / 6000;  // a launch, and the pieces' bytes out and in
    }
    return longest_pair(units, kb, count, pairs) * per_kb + fixed + (units[0] + units[1] - 1) / pairs * 500 + join;
  };
  int64_t cost = persistent(256, 270, 4700, false);
  LinPlan best = {256, 1};
  auto offer = [&](int64_t c, int tile, int S) {
    if (c >= cost) return false;
    cost = c;
    best = {tile, S};
    return true;
  };
  offer(persistent(128, 171, 3640, false), 128, 1);
  if (!g->b_mn) {
    offer(persistent(64, 171, 3300, false), 64, 1);
    const int64_t kb = (g->K + BK - 1) / BK, fit = max64(pairs * 36 / 76, 1);
    const int64_t tiles = (g->M + 255) / 256 * ((g->N + 127) / 128);
    if (kb >= 4) offer((tiles + fit - 1) / fit * ((kb + 1) / 2 * 180 + 7700), 128, 2);
  }
  bool pieces = false;
  for (int i = 0; i < count; ++i) pieces = pieces || g[i].pieces > 1;
  if (pieces) pieces = offer(persistent(256, 270, 4700, true), 256, 1);
  if (!pieces)
    for (int i = 0; i < count; ++i) g[i].pieces = 1;
  return best;
}

// The most K pieces of a weight gradient [N, K] over many tokens whose tiles leave pairs idle: as many as
// fill them, of 16 K blocks or more each (the workspace holds their fp32 products).
int wgrad_pieces(int64_t M, int64_t K, int64_t N) {
  const int64_t pairs = max64(num_sms() / 2, 1), tiles = ((N + 255) / 256) * ((K + 255) / 256), kb = (M + BK - 1) / BK;
  return (int)max64(1, min64(min64(8, pairs / max64(tiles, 1)), kb / 16));
}

// The forward of one token, and of two to four with few outputs, without a checkpoint (whose blocks span more columns
// than a warp has here; a decoding step keeps none). FMAs cost by the token and x is staged once a block; the form with
// tokens on the accumulator's columns costs the same up to 16 of them. us, this form and that (K x N): one token 4096 x 1024 3.3
// and 6.6, 4096 x 4096 7.8 and 9.0, 4096 x 14336 21.4 and 21.4; two 4096 x 4096 8.4 and 9.1, 4096 x 6144 13.8 and 12.2;
// four 4096 x 1024 5.3 and 6.7, 4096 x 2048 7.4 and 7.2, 4096 x 4096 10.2 and 9.2, 4096 x 14336 26.6 and 21.5.
bool takes_few(const LinGemm& g) {
  return g.M <= kFewTokens && (g.M == 1 || g.M * g.N <= kFewOutputs) && !g.a_mn && !g.b_mn && !g.ckpt.codes &&
         g.K * (g.M > 2 ? 4 : g.M) * 2 <= kFewMaxX;
}
template <int MT, bool F16>
lnfp8_status few_launch(const LinGemm& g, cudaStream_t st) {
  constexpr auto k = lin_few_kernel<MT, F16>;
  const lnfp8_status set = kernel_setup<k>(256, kFewMaxX, nullptr, "linear: kernel set-up");
  if (set != LNFP8_OK) return set;
  // warps per row group: until there are 8 warps for each SM, while each keeps 512 columns. One token, us with 1, 2, 4 and 8:
  // 1024 x 4096 3.2, 4.4, 6.7, 10.6; 4096 x 4096 7.8, 9.3, 10.9, 14.8; 8192 x 2048 9.2, 7.7, 9.1, 10.8;
  // 4096 x 1024 4.8, 3.7, 3.4, 4.7 (K x N; the rule takes 1, 1, 2, 4; until 16 warps it took one step more)
  int WK = 1;
  while (WK < 8 && (g.N + kRowsPerWarp - 1) / kRowsPerWarp * WK < (int64_t)num_sms() * 8 && g.K >= 1024 * WK) WK *= 2;
  const int64_t per_block = 8 / WK * kRowsPerWarp;
  LaunchScope ls("linear_few", st);
  if (launch_pdl(k, dim3((unsigned)((g.N + per_block - 1) / per_block)), dim3(256), (size_t)(MT * g.K * 2), st, epi_params(g), g.a, g.lda, g.b,
                 (int)g.K, WK) != cudaSuccess)
    return check_launch("linear launch");
  return check_launch("linear");
}
template <bool F16>
lnfp8_status few_by_tokens(const LinGemm& g, cudaStream_t st) {
  return g.M == 1 ? few_launch<1, F16>(g, st) : g.M == 2 ? few_launch<2, F16>(g, st) : few_launch<4, F16>(g, st);
}

// Few tokens: K pieces while they run on SMs that would idle and each keeps a few K blocks. 8 tokens, us with 1, 2 and 4
// pieces (K x N; 64 tokens within 5% the same way): 768 x 2304 5.0, 4.9, 4.6; 4096 x 1024 14.4, 9.4, 6.7; 4096 x 4096 14.9,
// 10.4, 9.3; 2048 x 8192 (two fill the SMs) 9.5, 9.1, 13.2; 4096 x 14336 (one fills them) 21.7, -, 34.3. The rule takes 4, 4,
// 4, 2 and 1; the one shape where it was not best is 64 x 1024 x 4096, 7.2, 6.6, 7.0.
int swap_splits(const LinGemm& g) {
  const int64_t tiles = (g.N + 127) / 128, kb = (g.K + BK - 1) / BK;
  int S = 1;
  while (S < 4 && tiles * S * 2 <= num_sms() && kb >= S * 2 * 2) S *= 2;
  return S;
}
lnfp8_status swap_launch(const LinGemm& g, cudaStream_t st) {
  const int S = swap_splits(g);
  return g.M <= 16 ? tile_launch<16, false, true>(g, S, st) : g.M <= 32 ? tile_launch<32, false, true>(g, S, st) : tile_launch<64, false, true>(g, S, st);
}
}  // namespace

lnfp8_status lin_gemm_launch(const LinGemm* g, int count, cudaStream_t st) {
  if (!g[0].b_mn) {  // the forward: both operands K-major
    if (g->M == 0 || g->N == 0) return LNFP8_OK;
    if (takes_few(*g)) return g->elem == LNFP8_FP16 ? few_by_tokens<true>(*g, st) : few_by_tokens<false>(*g, st);
    if (takes_swap(*g)) return swap_launch(*g, st);
    LinGemm one = *g;
    const LinPlan pl = lin_plan(&one, 1);
    if (pl.S == 2) return tile_launch<128, true, false>(*g, 2, st);
    return pl.tile == 64 ? pair_launch<64, LIN_FULL>(g, 1, st) : pl.tile == 128 ? pair_launch<128, LIN_FULL>(g, 1, st) : pair_launch<256, LIN_FULL>(g, 1, st);
  }
  // the backward: what few tokens leave swapped runs alone, the rest in one launch
  LinGemm rest[2];
  int n = 0;
  for (int i = 0; i < count; ++i) {
    if (!takes_swap(g[i])) {
      rest[n++] = g[i];
      continue;
    }
    const lnfp8_status s = swap_launch(g[i], st);
    if (s != LNFP8_OK) return s;
  }
  if (n == 0) return LNFP8_OK;
  const LinPlan pl = lin_plan(rest, n);
  lnfp8_status s = pl.tile == 128 ? pair_launch<128, LIN_PLAIN>(rest, n, st) : pair_launch<256, LIN_PLAIN>(rest, n, st);
  for (int i = 0; i < n && s == LNFP8_OK; ++i)
    if (rest[i].pieces > 1) s = join_launch(rest[i], st);
  return s;
}

lnfp8_status linear_act_fwd_launch(const lnfp8_linear_act_fwd_args* a, cudaStream_t st) {
  LinGemm g = {};
  g.M = a->M;
  g.N = a->N;
  g.K = a->K;
  g.elem = a->elem;
  g.a = a->x;
  g.lda = a->ldx;
  g.b = a->w;
  g.ldb = a->K;
  g.out = a->y;
  g.ldo = a->ldy;
  g.bias = a->bias;
  g.act = a->act;
  g.resid = a->residual;
  g.ldr = a->ld_residual;
  g.h = a->h;
  g.ckpt = a->ckpt;
  return lin_gemm_launch(&g, 1, st);
}

// dz [M, N], the restored x [M, K], two column sums for the affine input, the columns' partial sums and
// the K pieces of dw, each from a multiple of 256 on.
static int64_t wgrad_bytes(int64_t M, int64_t K, int64_t N) {
  const int pieces = wgrad_pieces(M, K, N);
  return pieces > 1 ? up256(pieces * N * K * 4) + 256 : 0;  // moved up to a 32-byte boundary
}
int64_t linear_act_bwd_ws_bytes(int64_t M, int64_t K, int64_t N, bool has_act, bool x_from_ckpt) {
  if (M == 0 || N == 0) return 0;
  const int64_t rpb = dact_rows_per_block(M, K, N, has_act);
  return (has_act ? up256(M * N * 2) : 0) + (x_from_ckpt ? up256(M * K * 2) + 2 * up256(N * 4) : 0) +
         up256((M + rpb - 1) / rpb * N * 4 * (has_act && x_from_ckpt ? 2 : 1)) + wgrad_bytes(M, K, N);
}

lnfp8_status linear_act_bwd_launch(const lnfp8_linear_act_bwd_args* a, cudaStream_t st) {
  if (a->M == 0) {
    if ((a->dw && cudaMemsetAsync(a->dw, 0, a->N * a->K * 2, st) != cudaSuccess) ||
        (a->dbias && cudaMemsetAsync(a->dbias, 0, a->N * sizeof(float), st) != cudaSuccess))
      return check_launch("linear_act_bwd: clearing dw/dbias");
    return LNFP8_OK;
  }
  const bool has_act = a->act != LNFP8_ACT_NONE, xck = a->x_ckpt.codes != nullptr;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  void* dz_ws = ws;
  if (has_act) ws += up256(a->M * a->N * 2);
  void* x_ws = ws;
  if (xck) ws += up256(a->M * a->K * 2);
  // x = v gamma + beta from a checkpoint's values v: dw = (dz^T v) gamma + (sum dz) beta, applied in the
  // product's epilogue, and x is never formed or rounded. v has at most four significant bits: a bf16 operand holds it
  // exactly, an fp16 one where it lies in fp16's range (past 65504 it saturates, and below 2^-14 it keeps steps of 2^-24,
  // which the smallest codes do not reach in E4M3 blocks whose largest value is under 0.007 and in E5M2 blocks under
  // 112). The sum is of dz as rounded for the product, so that where v gamma and beta cancel, dw does too.
  const bool affine = a->dw && xck && a->x_gamma;
  float* db = a->dbias;
  float* dbr = nullptr;
  if (xck) {
    if (affine) {
      if (!db) db = reinterpret_cast<float*>(ws);
      dbr = has_act ? reinterpret_cast<float*>(ws + up256(a->N * 4)) : db;
    }
    ws += 2 * up256(a->N * 4);
  }
  const void* dz = has_act ? dz_ws : a->dy;
  const int64_t lddz = has_act ? a->N : a->ld_dy;

  if (has_act || db) {
    DactParams p;
    p.dy = a->dy;
    p.h = a->h;
    p.codes = a->h_ckpt.codes;
    p.scales = a->h_ckpt.scales;
    p.dz = dz_ws;
    const bool few_rows = a->M <= dact_cluster_rows(a->K, a->N, has_act), clustered = db && few_rows;
    p.part = db && !clustered ? reinterpret_cast<float*>(ws) : nullptr;
    p.db = clustered ? db : nullptr;
    p.dbr = dbr;
    p.both = affine && has_act;
    p.M = a->M;
    p.lddy = a->ld_dy;
    p.pitch = lnfp8_act_ckpt_scale_pitch(a->N);
    p.N = (int)a->N;
    p.dt = a->h_ckpt.dtype;
    p.rows_per_block = (int)dact_rows_per_block(a->M, a->K, a->N, has_act);
    const int64_t row_blocks = few_rows ? kDactCluster : (a->M + p.rows_per_block - 1) / p.rows_per_block;
    const dim3 grid((unsigned)((a->N + 255) / 256), (unsigned)row_blocks);
    auto pick = [&](auto elem) {
      constexpr int E = decltype(elem)::value;
      if (!has_act) return dact_launch<E, DACT_NONE, LNFP8_ACT_NONE>(p, grid, st);
      if (p.codes)
        return a->act == LNFP8_ACT_GELU   ? dact_launch<E, DACT_CKPT, LNFP8_ACT_GELU>(p, grid, st)
               : a->act == LNFP8_ACT_SILU ? dact_launch<E, DACT_CKPT, LNFP8_ACT_SILU>(p, grid, st)
                                          : dact_launch<E, DACT_CKPT, LNFP8_ACT_RELU>(p, grid, st);
      return a->act == LNFP8_ACT_GELU   ? dact_launch<E, DACT_TENSOR, LNFP8_ACT_GELU>(p, grid, st)
             : a->act == LNFP8_ACT_SILU ? dact_launch<E, DACT_TENSOR, LNFP8_ACT_SILU>(p, grid, st)
                                        : dact_launch<E, DACT_TENSOR, LNFP8_ACT_RELU>(p, grid, st);
    };
    lnfp8_status s = a->elem == LNFP8_BF16 ? pick(std::integral_constant<int, LNFP8_BF16>()) : pick(std::integral_constant<int, LNFP8_FP16>());
    if (s != LNFP8_OK) return s;
    if (p.part) {
      s = colsum_launch(p.part, (int)row_blocks, p.N * (1 + p.both), p.N, db, dbr, st);
      if (s != LNFP8_OK) return s;
    }
  }
  LinGemm g[2] = {};
  int count = 0;
  if (a->dx) {  // [M, K] = dz [M, N] . w, contracted over N
    LinGemm& q = g[count++];
    q.elem = a->elem;
    q.M = a->M;
    q.N = a->K;
    q.K = a->N;
    q.a = dz;
    q.lda = lddz;
    q.b = a->w;
    q.ldb = a->K;
    q.b_mn = true;
    q.out = a->dx;
    q.ldo = a->ld_dx;
  }
  if (a->dw) {  // [N, K] = dz^T . x, contracted over the tokens
    LinGemm& q = g[count++];
    q.elem = a->elem;
    q.b = a->x;
    q.ldb = a->ldx;
    if (xck) {
      const lnfp8_status s = act_ckpt_restore_launch(a->x_ckpt, a->M, a->K, a->x_act, nullptr, nullptr, a->elem, x_ws, a->elem, a->K, st);
      if (s != LNFP8_OK) return s;
      q.b = x_ws;
      q.ldb = a->K;
    }
    q.M = a->N;
    q.N = a->K;
    q.K = a->M;
    q.a = dz;
    q.lda = lddz;
    q.a_mn = true;
    q.b_mn = true;
    q.out = a->dw;
    q.ldo = a->K;
    q.pieces = wgrad_pieces(a->M, a->K, a->N);
    if (q.pieces > 1) {  // the last part of the workspace
      const uintptr_t at = reinterpret_cast<uintptr_t>(a->workspace) + linear_act_bwd_ws_bytes(a->M, a->K, a->N, has_act, xck) -
                           wgrad_bytes(a->M, a->K, a->N);
      q.part = reinterpret_cast<float*>((at + 31) / 32 * 32);
    }
    if (affine) {
      q.cscale = a->x_gamma;
      q.cvec = a->x_beta;
      q.rvec = dbr;
    }
  }
  return count ? lin_gemm_launch(g, count, st) : LNFP8_OK;
}

}  // namespace lnfp8
