// 8-bit activation checkpoints: save (16- or 32-bit tensor -> FP8 codes and one
// power-of-two scale per 32 columns of a row) and restore (codes -> 16- or 32-bit
// values, optionally through an activation or a per-column gamma, beta). The
// block format is described in rowmath.cuh. Activations are what a training step
// keeps most of (TE tutorial, code block 4: the peak-memory comparison); the FP8
// codes halve them against bf16 without touching the delayed-scaling state.
#include "common.cuh"
#include "internal.h"
#include "rowmath.cuh"

namespace lnfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerWarp = 8;  // checkpoint blocks a warp takes per step, for loads in flight

struct SaveParams {
  const void* x;
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, ldx, pitch, units;  // units: rows * ceil(blocks per row / kBlocksPerWarp)
  int cols, upr;                    // upr: units per row
};

struct RestoreParams {
  const uint8_t* codes;
  const uint8_t* scales;
  const void* gamma;
  const void* beta;
  void* out;
  int64_t rows, ldo, pitch, units;
  int cols, upr, act, param_elem;
};

// Any width and alignment: a warp takes kBlocksPerWarp blocks of a row, lane = column.
template <int ELEM, int DT>
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
      const uint32_t b = ckpt_byte<DT>(warp_max_u32(abs_bits(v[i])));
      const uint16_t code = cvt_fp8x2<DT>(v[i] * ckpt_inv_scale(b), 0.f);
      if (c < p.cols) {
        p.codes[row * p.cols + c] = (uint8_t)code;
        if (lane == 0) p.scales[row * p.pitch + (c >> 5)] = (uint8_t)b;
      }
    }
  }
}

template <int ELEM, int DT>
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
      float v = fp8x2_to_f32<DT>(code[i]).x * ckpt_scale(byte[i]);
      if (p.gamma) v = fmaf(v, load_elem_rt(p.gamma, p.param_elem, c), load_elem_rt(p.beta, p.param_elem, c));
      store_elem<ELEM>(p.out, row * p.ldo + c, ckpt_clamp<ELEM>(act_fwd(v, p.act)));
    }
  }
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
  p.cols = (int)cols;
  p.upr = (int)((cols + kBlocksPerWarp * 32 - 1) / (kBlocksPerWarp * 32));
  p.units = rows * p.upr;
  LaunchScope ls("act_ckpt_save", st);
  auto go = [&](auto kernel) {
    if (launch_pdl(kernel, dim3(grid_for(p.units)), dim3(kThreads), 0, st, p) != cudaSuccess) return check_launch("act_ckpt_save launch");
    return check_launch("act_ckpt_save");
  };
  const bool e4 = c.dtype == LNFP8_E4M3;
  if (elem == LNFP8_BF16) return e4 ? go(save_any_kernel<LNFP8_BF16, LNFP8_E4M3>) : go(save_any_kernel<LNFP8_BF16, LNFP8_E5M2>);
  if (elem == LNFP8_FP16) return e4 ? go(save_any_kernel<LNFP8_FP16, LNFP8_E4M3>) : go(save_any_kernel<LNFP8_FP16, LNFP8_E5M2>);
  return e4 ? go(save_any_kernel<LNFP8_FP32, LNFP8_E4M3>) : go(save_any_kernel<LNFP8_FP32, LNFP8_E5M2>);
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
  const bool e4 = c.dtype == LNFP8_E4M3;
  if (elem == LNFP8_BF16) return e4 ? go(restore_any_kernel<LNFP8_BF16, LNFP8_E4M3>) : go(restore_any_kernel<LNFP8_BF16, LNFP8_E5M2>);
  if (elem == LNFP8_FP16) return e4 ? go(restore_any_kernel<LNFP8_FP16, LNFP8_E4M3>) : go(restore_any_kernel<LNFP8_FP16, LNFP8_E5M2>);
  return e4 ? go(restore_any_kernel<LNFP8_FP32, LNFP8_E4M3>) : go(restore_any_kernel<LNFP8_FP32, LNFP8_E5M2>);
}

}  // namespace lnfp8
