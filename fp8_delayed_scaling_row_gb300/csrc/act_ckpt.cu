// 8-bit activation checkpoints: save (16- or 32-bit tensor -> FP8 codes and one
// power-of-two scale per 32 columns of a row) and restore (codes -> 16- or 32-bit
// values, optionally through an activation or a per-column gamma, beta). The
// block format is described in rowmath.cuh. Activations are what a training step
// keeps most of (TE tutorial, code block 4: the peak-memory comparison); the FP8
// codes halve them against bf16 without touching the delayed-scaling state.
#include "common.cuh"
#include "internal.h"
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
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < p.units; u += warps) {
    const int64_t row = u / p.upr;
    const int c0 = (int)(u - row * p.upr) * (kBlocksPerWarp * 32) + lane;
    float v[kBlocksPerWarp];
#pragma unroll
    for (int i = 0; i < kBlocksPerWarp; ++i) v[i] = c0 + 32 * i < p.cols ? load_elem<ELEM>(p.x, row * p.ldx + c0 + 32 * i) : 0.f;
#pragma unroll
    for (int i = 0; i < kBlocksPerWarp; ++i) {
      const int c = c0 + 32 * i;
      const uint32_t b = ckpt_byte(warp_max_u32(abs_bits(v[i])), p.dt);
      const uint32_t code = fp8x2(v[i] * ckpt_inv_scale(b), 0.f, p.dt);
      if (c < p.cols) {
        p.codes[row * p.cols + c] = (uint8_t)code;
        if (lane == 0) p.scales[row * p.pitch + (c >> 5)] = (uint8_t)b;
      }
    }
  }
}

template <int ELEM>
__global__ void __launch_bounds__(kThreads) restore_any_kernel(const RestoreParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < p.units; u += warps) {
    const int64_t row = u / p.upr;
    const int c0 = (int)(u - row * p.upr) * (kBlocksPerWarp * 32) + lane;
    uint32_t code[kBlocksPerWarp], byte[kBlocksPerWarp];
#pragma unroll
    for (int i = 0; i < kBlocksPerWarp; ++i) {
      const int c = c0 + 32 * i;
      code[i] = c < p.cols ? p.codes[row * p.cols + c] : 0u;
      byte[i] = c < p.cols ? p.scales[row * p.pitch + (c >> 5)] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kBlocksPerWarp; ++i) {
      const int c = c0 + 32 * i;
      if (c >= p.cols) continue;
      float v = fp8x2_to_f32(code[i], p.dt).x * ckpt_scale(byte[i]);
      if (p.gamma) v = fmaf(v, load_elem_rt(p.gamma, p.param_elem, c), load_elem_rt(p.beta, p.param_elem, c));
      store_elem<ELEM>(p.out, row * p.ldo + c, ckpt_clamp<ELEM>(act_fwd(v, p.act)));
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
      // values past the type's range: with gamma and beta anywhere, else in blocks of large scales only
      if (AFFINE || b[k] >= (ELEM == LNFP8_FP16 ? 127u : 239u)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 t = upk(v[e]);
          v[e] = pk(ckpt_clamp<ELEM>(t.x), ckpt_clamp<ELEM>(t.y));
        }
      }
      store8<ELEM>(p.out, row[k] * p.ldo + col[k], v);
    }
  }
}

bool al(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

unsigned vec_grid(int64_t chunks) {
  const int64_t blocks = (chunks + kThreads * kChunks - 1) / (kThreads * kChunks);
  return (unsigned)max64(1, min64(blocks, (int64_t)num_sms() * 8));
}

unsigned grid_for(int64_t warps_of_work) {
  const int64_t blocks = (warps_of_work + kThreads / 32 - 1) / (kThreads / 32);
  return (unsigned)max64(1, min64(blocks, (int64_t)num_sms() * (2048 / kThreads)));
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
  auto go = [&](auto kernel) {
    if (launch_pdl(kernel, dim3(grid_for(p.units)), dim3(kThreads), 0, st, p) != cudaSuccess) return check_launch("act_ckpt_save launch");
    return check_launch("act_ckpt_save");
  };
  // 16-byte rows take the vector kernel
  if (cols % 8 == 0 && al(x, 16) && ldx * (elem == LNFP8_FP32 ? 4 : 2) % 16 == 0 && al(c.codes, 8)) {
    p.upr = (int)((cols + 31) / 32 * 4);
    const unsigned grid = vec_grid(rows * p.upr);
    p.row_step = (int64_t)grid * kThreads / p.upr;
    p.chunk_step = (uint32_t)((int64_t)grid * kThreads % p.upr);
    auto vec = [&](auto kernel) {
      if (launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, st, p) != cudaSuccess) return check_launch("act_ckpt_save launch");
      return check_launch("act_ckpt_save");
    };
    if (elem == LNFP8_BF16) return vec(save_vec_kernel<LNFP8_BF16>);
    return elem == LNFP8_FP16 ? vec(save_vec_kernel<LNFP8_FP16>) : vec(save_vec_kernel<LNFP8_FP32>);
  }
  if (elem == LNFP8_BF16) return go(save_any_kernel<LNFP8_BF16>);
  return elem == LNFP8_FP16 ? go(save_any_kernel<LNFP8_FP16>) : go(save_any_kernel<LNFP8_FP32>);
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
  auto go = [&](auto kernel) {
    if (launch_pdl(kernel, dim3(grid_for(p.units)), dim3(kThreads), 0, st, p) != cudaSuccess) return check_launch("act_ckpt_restore launch");
    return check_launch("act_ckpt_restore");
  };
  if (cols % 8 == 0 && al(out, 16) && ldo * (elem == LNFP8_FP32 ? 4 : 2) % 16 == 0 && al(c.codes, 8) &&
      (!gamma || (al(gamma, 16) && al(beta, 16)))) {
    p.upr = (int)((cols + 31) / 32 * 4);
    const unsigned grid = vec_grid(rows * p.upr);
    p.row_step = (int64_t)grid * kThreads / p.upr;
    p.chunk_step = (uint32_t)((int64_t)grid * kThreads % p.upr);
    auto vec = [&](auto kernel) {
      if (launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, st, p) != cudaSuccess) return check_launch("act_ckpt_restore launch");
      return check_launch("act_ckpt_restore");
    };
    auto by_act = [&](auto e) {
      constexpr int E = decltype(e)::value;
      if (gamma) return vec(restore_vec_kernel<E, LNFP8_ACT_NONE, true>);
      if (act == LNFP8_ACT_GELU) return vec(restore_vec_kernel<E, LNFP8_ACT_GELU, false>);
      if (act == LNFP8_ACT_SILU) return vec(restore_vec_kernel<E, LNFP8_ACT_SILU, false>);
      return act == LNFP8_ACT_RELU ? vec(restore_vec_kernel<E, LNFP8_ACT_RELU, false>) : vec(restore_vec_kernel<E, LNFP8_ACT_NONE, false>);
    };
    if (elem == LNFP8_BF16) return by_act(std::integral_constant<int, LNFP8_BF16>());
    return elem == LNFP8_FP16 ? by_act(std::integral_constant<int, LNFP8_FP16>()) : by_act(std::integral_constant<int, LNFP8_FP32>());
  }
  if (elem == LNFP8_BF16) return go(restore_any_kernel<LNFP8_BF16>);
  return elem == LNFP8_FP16 ? go(restore_any_kernel<LNFP8_FP16>) : go(restore_any_kernel<LNFP8_FP32>);
}

}  // namespace lnfp8
