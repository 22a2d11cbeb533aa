// Sums over the threads that share a row, for the kernels that give a row to a group of TPR threads
// (layernorm_rows.cu, block_join_fwd.cu, block_join_bwd.cu).
#pragma once

#include "common.cuh"

namespace lnfp8 {

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

}  // namespace lnfp8
