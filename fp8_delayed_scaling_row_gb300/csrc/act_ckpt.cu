// 8-bit activation checkpoints: save (16- or 32-bit tensor -> FP8 codes and one
// power-of-two scale per 32 columns of a row) and restore (codes -> 16- or 32-bit
// values, optionally through an activation or a per-column gamma, beta). The
// block format is described in rowmath.cuh. Activations are what a training step
// keeps most of (TE tutorial, code block 4: the peak-memory comparison); the FP8
// codes halve them against bf16 without touching the delayed-scaling state.
#include "common.cuh"
#include "internal.h"
#include "kernel_setup.cuh"
#include "rowmath.cuh"

#include <type_traits>

namespace lnfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerWarp = 8;  // checkpoint blocks a warp takes per step, for loads in flight

struct SaveParams {
  const void* x;
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, ldx, pitch, units;  // units: rows * ceil(blocks per row / kBlocksPerWarp)
  int cols, upr, dt;                // upr: units per row; dt: the lnfp8_dtype of the codes
  int64_t row_step;                 // chunks of a pass over the grid, in rows and chunks
  uint32_t chunk_step;
};

struct RestoreParams {
  const uint8_t* codes;
  const uint8_t* scales;
  const void* gamma;
  const void* beta;
  void* out;
  int64_t rows, ldo, pitch, units;
  int cols, upr, act, param_elem, dt;
  int64_t row_step;
  uint32_t chunk_step;
};

// Any width and alignment: a warp takes kBlocksPerWarp blocks of a row, lane = column.
template <int ELEM>
__global__ void __launch_bounds__(kThreads) save_any_kernel(const SaveParams p) {
  constexpr int ES = ElemSize<ELEM>::value;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < p.units; u += warps) {
    const int64_t row = u / p.upr;
    const int c0 = (int)(u - row * p.upr) * (kBlocksPerWarp * 32) + lane;
    const int left = p.cols - c0;  // block i of this lane is inside while 32 i < left
    const uint8_t* src = static_cast<const uint8_t*>(p.x) + (row * p.ldx + c0) * ES;
    uint8_t *cd = p.codes + row * p.cols + c0, *sc = p.scales + row * p.pitch + (c0 >> 5);
    float v[kBlocksPerWarp];
#pragma unroll
    for (int i = 0; i < kBlocksPerWarp; ++i) v[i] = 32 * i < left ? load_elem<ELEM>(src, 32 * i) : 0.f;
#pragma unroll
    for (int i = 0; i < kBlocksPerWarp; ++i) {
      const uint32_t b = ckpt_byte(__reduce_max_sync(0xFFFFFFFFu, abs_bits(v[i])), p.dt);
      const uint32_t code = fp8x2(v[i] * ckpt_inv_scale(b), 0.f, p.dt);
      if (32 * i < left) {
        cd[32 * i] = (uint8_t)code;
        if (lane == 0) sc[i] = (uint8_t)b;
      }
    }
  }
}

template <int ELEM>
__global__ void __launch_bounds__(kThreads) restore_any_kernel(const RestoreParams p) {
  constexpr int ES = ElemSize<ELEM>::value;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < p.units; u += warps) {
    const int64_t row = u / p.upr;
    const int c0 = (int)(u - row * p.upr) * (kBlocksPerWarp * 32) + lane;
    const int left = p.cols - c0;
    const uint8_t *cd = p.codes + row * p.cols + c0, *sc = p.scales + row * p.pitch + (c0 >> 5);
    uint8_t* dst = static_cast<uint8_t*>(p.out) + (row * p.ldo + c0) * ES;
    uint32_t code[kBlocksPerWarp], byte[kBlocksPerWarp];
#pragma unroll
    for (int i = 0; i < kBlocksPerWarp; ++i) {
      code[i] = 32 * i < left ? cd[32 * i] : 0u;
      byte[i] = 32 * i < left ? sc[i] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kBlocksPerWarp; ++i) {
      if (32 * i >= left) break;
      float v = fp8x2_to_f32(code[i], p.dt).x * ckpt_scale(byte[i]);
      if (p.gamma) v = fmaf(v, load_elem_rt(p.gamma, p.param_elem, c0 + 32 * i), load_elem_rt(p.beta, p.param_elem, c0 + 32 * i));
      store_elem<ELEM>(dst, 32 * i, ckpt_clamp<ELEM>(act_fwd(v, p.act)));
    }
  }
}

// Rows of whole 8-element chunks on 16-byte boundaries: a thread takes kChunks chunks of 8, a warp's
// lanes neighbouring ones, so that four lanes hold a block. Chunks are counted over the rows with
// each row's last block padded to 32 columns (cpr chunks a row), which keeps blocks inside four lanes.
// HBM-bound: kChunks independent 16-byte loads a thread cover the latency.
constexpr int kChunks = 4;

// The place of a chunk, moved on by a fixed number of chunks at a time (one division in all).
struct ChunkPlace {
  int64_t row;
  uint32_t c;  // chunk within the row
  __device__ __forceinline__ ChunkPlace(int64_t chunk, uint32_t cpr) {
    row = chunk / cpr;
    c = (uint32_t)(chunk - row * cpr);
  }
  __device__ __forceinline__ void move(int64_t rows, uint32_t chunks, uint32_t cpr) {
    row += rows;
    c += chunks;
    if (c >= cpr) {
      c -= cpr;
      ++row;
    }
  }
};

template <int ELEM>
__global__ void __launch_bounds__(kThreads) save_vec_kernel(const SaveParams p) {
  constexpr int W = ELEM == LNFP8_FP32 ? 2 : 1;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t step = (int64_t)gridDim.x * kThreads;
  const uint32_t cpr = p.upr;  // chunks per row here
  int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  ChunkPlace at(i, cpr);
  const int64_t end = (p.rows * cpr + 31) / 32 * 32;  // whole warps reach the shuffles
  while (i < end) {
    uint4 u[kChunks][W];
    int64_t row[kChunks];
    int col[kChunks];  // -1: past the row's or the tensor's end
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      row[k] = at.row;
      col[k] = at.row < p.rows && (int)at.c * 8 < p.cols ? (int)at.c * 8 : -1;
#pragma unroll
      for (int w = 0; w < W; ++w) u[k][w] = make_uint4(0u, 0u, 0u, 0u);
      if (col[k] >= 0) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + (at.row * p.ldx + col[k]) * ElemSize<ELEM>::value);
#pragma unroll
        for (int w = 0; w < W; ++w) u[k][w] = __ldcs(src + w);
      }
      at.move(p.row_step, p.chunk_step, cpr);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      if (i + k * step >= end) break;  // uniform over the warp
      uint64_t v[4];
      unpack8<ELEM>(u[k], v);
      const uint32_t b = ckpt_byte(block_amax8(v), p.dt);
      if (col[k] >= 0) {
        *reinterpret_cast<uint2*>(p.codes + row[k] * p.cols + col[k]) = encode8(v, ckpt_inv_scale(b), p.dt);
        if ((col[k] & 31) == 0) p.scales[row[k] * p.pitch + (col[k] >> 5)] = (uint8_t)b;
      }
    }
    i += kChunks * step;
  }
}

// Values past the type's range (those of blocks of large scales only; no activation enlarges one).
template <int ELEM>
__device__ __forceinline__ void restore_clamp(uint32_t b, uint64_t* v) {
  if (b < (ELEM == LNFP8_FP16 ? 127u : 239u)) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 t = upk(v[e]);
    v[e] = pk(ckpt_clamp<ELEM>(t.x), ckpt_clamp<ELEM>(t.y));
  }
}

template <int ELEM, int ACT, bool AFFINE>
__global__ void __launch_bounds__(kThreads) restore_vec_kernel(const RestoreParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t cpr = p.upr;
  ChunkPlace at((int64_t)blockIdx.x * kThreads + threadIdx.x, cpr);
  while (at.row < p.rows) {
    uint2 q[kChunks];
    uint32_t b[kChunks];
    int64_t row[kChunks];
    int col[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      row[k] = at.row;
      col[k] = at.row < p.rows && (int)at.c * 8 < p.cols ? (int)at.c * 8 : -1;
      q[k] = make_uint2(0u, 0u);
      b[k] = 0u;
      if (col[k] >= 0) {
        q[k] = __ldcs(reinterpret_cast<const uint2*>(p.codes + at.row * p.cols + col[k]));
        b[k] = __ldg(p.scales + at.row * p.pitch + (at.c >> 2));
      }
      at.move(p.row_step, p.chunk_step, cpr);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      if (col[k] < 0) continue;
      uint64_t v[4];
      decode8(q[k], ckpt_scale(b[k]), p.dt, v);
      if constexpr (AFFINE) {
        uint64_t ga[4], be[4];
        load8_rt(p.gamma, p.param_elem, col[k], ga);
        load8_rt(p.beta, p.param_elem, col[k], be);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fma_2(v[e], ga[e], be[e]);
      }
      act8<ACT>(v);
      restore_clamp<ELEM>(AFFINE ? 255u : b[k], v);
      store8<ELEM>(p.out, row[k] * p.ldo + col[k], v);
    }
  }
}

// A tensor of contiguous rows of whole 128 columns is one long row, scales and all: chunk i has its codes at
// 8 i and its scale at i / 4. A block takes tiles of kChunks x 256 chunks, a thread every 256th of a
// tile, so that a tile costs a pointer step each and no index arithmetic (restore of 16384 x 8192 with GELU
// 86 us with places, 67 flat).
constexpr int kTile = kThreads * kChunks;

template <int ELEM>
__global__ void __launch_bounds__(kThreads) save_flat_kernel(const SaveParams p, const int64_t chunks) {
  constexpr int W = ELEM == LNFP8_FP32 ? 2 : 1, ES = ElemSize<ELEM>::value;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t base = (int64_t)blockIdx.x * kTile; base < chunks; base += (int64_t)gridDim.x * kTile) {
    const int64_t first = base + threadIdx.x;
    const uint8_t* src = static_cast<const uint8_t*>(p.x) + first * 8 * ES;
    uint8_t *cd = p.codes + first * 8, *sc = p.scales + (first >> 2);
    const int left = (int)min64(chunks - base, kTile);  // a multiple of 16: whole rows
    uint4 u[kChunks][W];
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        u[k][w] = make_uint4(0u, 0u, 0u, 0u);
        if ((int)threadIdx.x + k * kThreads < left) u[k][w] = __ldcs(reinterpret_cast<const uint4*>(src + k * kThreads * 8 * ES) + w);
      }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      uint64_t v[4];
      unpack8<ELEM>(u[k], v);
      const uint32_t b = ckpt_byte(block_amax8(v), p.dt);
      if ((int)threadIdx.x + k * kThreads < left) {
        *reinterpret_cast<uint2*>(cd + k * kThreads * 8) = encode8(v, ckpt_inv_scale(b), p.dt);
        if ((threadIdx.x & 3) == 0) sc[k * kThreads / 4] = (uint8_t)b;
      }
    }
  }
}

template <int ELEM, int ACT>
__global__ void __launch_bounds__(kThreads) restore_flat_kernel(const RestoreParams p, const int64_t chunks) {
  constexpr int ES = ElemSize<ELEM>::value;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t base = (int64_t)blockIdx.x * kTile; base < chunks; base += (int64_t)gridDim.x * kTile) {
    const int64_t first = base + threadIdx.x;
    const uint8_t *cd = p.codes + first * 8, *sc = p.scales + (first >> 2);
    uint8_t* dst = static_cast<uint8_t*>(p.out) + first * 8 * ES;
    const int left = (int)min64(chunks - base, kTile);
    uint2 q[kChunks];
    uint32_t b[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
      if ((int)threadIdx.x + k * kThreads < left) {
        q[k] = __ldcs(reinterpret_cast<const uint2*>(cd + k * kThreads * 8));
        b[k] = __ldg(sc + k * kThreads / 4);
      }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      if ((int)threadIdx.x + k * kThreads >= left) break;
      uint64_t v[4];
      decode8(q[k], ckpt_scale(b[k]), p.dt, v);
      act8<ACT>(v);
      restore_clamp<ELEM>(b[k], v);
      store8<ELEM>(dst, k * kThreads * 8, v);
    }
  }
}

bool al(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// One wave of resident blocks at most: a second, partial one would leave SMs idle at the end.
template <auto Kernel, typename... Args>
lnfp8_status run(int64_t blocks, cudaStream_t st, const char* who, Args... args) {
  int bps = 1;
  const lnfp8_status s = kernel_setup<Kernel>(kThreads, 0, &bps, who);
  if (s != LNFP8_OK) return s;
  const int64_t grid = max64(1, min64(blocks, (int64_t)num_sms() * bps));
  if (launch_pdl(Kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, args...) != cudaSuccess) return check_launch(who);
  return check_launch(who);
}
// The same for the kernels that move by places: their step over the grid in rows and chunks.
template <auto Kernel, typename P>
lnfp8_status run_places(P p, cudaStream_t st, const char* who) {
  int bps = 1;
  const lnfp8_status s = kernel_setup<Kernel>(kThreads, 0, &bps, who);
  if (s != LNFP8_OK) return s;
  p.upr = (p.cols + 31) / 32 * 4;
  const int64_t per = (int64_t)kThreads * kChunks;
  const int64_t grid = max64(1, min64((p.rows * p.upr + per - 1) / per, (int64_t)num_sms() * bps));
  p.row_step = grid * kThreads / p.upr;
  p.chunk_step = (uint32_t)(grid * kThreads % p.upr);
  if (launch_pdl(Kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, p) != cudaSuccess) return check_launch(who);
  return check_launch(who);
}

}  // namespace

lnfp8_status act_ckpt_save_launch(const void* x, int elem, int64_t rows, int64_t cols, int64_t ldx, const lnfp8_ckpt& c,
                                  cudaStream_t st) {
  if (rows == 0) return LNFP8_OK;
  SaveParams p;
  p.x = x;
  p.codes = c.codes;
  p.scales = c.scales;
  p.rows = rows;
  p.ldx = ldx;
  p.pitch = lnfp8_act_ckpt_scale_pitch(cols);
  p.dt = c.dtype;
  p.cols = (int)cols;
  p.upr = (int)((cols + kBlocksPerWarp * 32 - 1) / (kBlocksPerWarp * 32));
  p.units = rows * p.upr;
  LaunchScope ls("act_ckpt_save", st);
  const char* who = "act_ckpt_save";
  const int es = elem == LNFP8_FP32 ? 4 : 2;
  auto by_elem = [&](auto e) {
    constexpr int E = decltype(e)::value;
    if (cols % 128 == 0 && ldx == cols && al(x, 16) && al(c.codes, 8)) {
      const int64_t chunks = rows * cols / 8;
      return run<save_flat_kernel<E>>((chunks + kTile - 1) / kTile, st, who, p, chunks);
    }
    if (cols % 8 == 0 && al(x, 16) && ldx * es % 16 == 0 && al(c.codes, 8)) return run_places<save_vec_kernel<E>>(p, st, who);
    return run<save_any_kernel<E>>((p.units + kThreads / 32 - 1) / (kThreads / 32), st, who, p);
  };
  if (elem == LNFP8_BF16) return by_elem(std::integral_constant<int, LNFP8_BF16>());
  return elem == LNFP8_FP16 ? by_elem(std::integral_constant<int, LNFP8_FP16>()) : by_elem(std::integral_constant<int, LNFP8_FP32>());
}

lnfp8_status act_ckpt_restore_launch(const lnfp8_ckpt& c, int64_t rows, int64_t cols, int act, const void* gamma,
                                     const void* beta, int param_elem, void* out, int elem, int64_t ldo, cudaStream_t st) {
  if (rows == 0) return LNFP8_OK;
  RestoreParams p;
  p.codes = c.codes;
  p.scales = c.scales;
  p.gamma = gamma;
  p.beta = beta;
  p.out = out;
  p.rows = rows;
  p.ldo = ldo;
  p.pitch = lnfp8_act_ckpt_scale_pitch(cols);
  p.dt = c.dtype;
  p.cols = (int)cols;
  p.upr = (int)((cols + kBlocksPerWarp * 32 - 1) / (kBlocksPerWarp * 32));
  p.units = rows * p.upr;
  p.act = act;
  p.param_elem = param_elem;
  LaunchScope ls("act_ckpt_restore", st);
  const char* who = "act_ckpt_restore";
  const int es = elem == LNFP8_FP32 ? 4 : 2;
  const bool vec = cols % 8 == 0 && al(out, 16) && ldo * es % 16 == 0 && al(c.codes, 8) && (!gamma || (al(gamma, 16) && al(beta, 16)));
  auto by_act = [&](auto e, auto a) {
    constexpr int E = decltype(e)::value, A = decltype(a)::value;
    if (vec && cols % 128 == 0 && ldo == cols) {
      const int64_t chunks = rows * cols / 8;
      return run<restore_flat_kernel<E, A>>((chunks + kTile - 1) / kTile, st, who, p, chunks);
    }
    return run_places<restore_vec_kernel<E, A, false>>(p, st, who);
  };
  auto by_elem = [&](auto e) {
    constexpr int E = decltype(e)::value;
    if (!vec) return run<restore_any_kernel<E>>((p.units + kThreads / 32 - 1) / (kThreads / 32), st, who, p);
    if (gamma) return run_places<restore_vec_kernel<E, LNFP8_ACT_NONE, true>>(p, st, who);
    if (act == LNFP8_ACT_GELU) return by_act(e, std::integral_constant<int, LNFP8_ACT_GELU>());
    if (act == LNFP8_ACT_SILU) return by_act(e, std::integral_constant<int, LNFP8_ACT_SILU>());
    return act == LNFP8_ACT_RELU ? by_act(e, std::integral_constant<int, LNFP8_ACT_RELU>()) : by_act(e, std::integral_constant<int, LNFP8_ACT_NONE>());
  };
  if (elem == LNFP8_BF16) return by_elem(std::integral_constant<int, LNFP8_BF16>());
  return elem == LNFP8_FP16 ? by_elem(std::integral_constant<int, LNFP8_FP16>()) : by_elem(std::integral_constant<int, LNFP8_FP32>());
}

}  // namespace lnfp8
