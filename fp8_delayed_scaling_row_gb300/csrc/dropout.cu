// Dropout whose mask is never stored: y = x / (1 - p) where the element's draw keeps it, else 0. The backward is the
// same map on the gradient. Bound by HBM: an element is read once and written once.
#include "common.cuh"
#include "internal.h"
#include "kernel_setup.cuh"
#include "philox.cuh"
#include "rowmath.cuh"

namespace lnfp8 {
namespace {

struct DropoutParams {
  const void* x;
  void* y;
  int64_t rows, ldx, ldy;
  int cols;
  float scale;
  DropParams drop;
  int64_t step_rows;  // what a thread's next item lies ahead: rows, and groups of eight columns
  uint32_t step_groups;
};

constexpr int kDropWarps = 8;

// Any width and alignment: a warp takes 256 columns of a row. Lane q draws for the q-th group of eight, and the draws go
// through shared memory to the lanes that hold the columns (32 neighbours at a time).
template <int ELEM>
__global__ void __launch_bounds__(32 * kDropWarps) dropout_any_kernel(const DropoutParams p) {
  __shared__ __align__(16) uint16_t bits[kDropWarps][256];
  pdl_wait();
  pdl_launch_dependents();
  drop_save(p.drop);
  const DropKey key = drop_key(p.drop);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t parts = (p.cols + 255) / 256, total = p.rows * parts;
  for (int64_t i = (int64_t)blockIdx.x * kDropWarps + w; i < total; i += (int64_t)gridDim.x * kDropWarps) {
    const int64_t row = i / parts;
    const int c0 = (int)(i - row * parts) * 256;
    const int64_t xo = row * p.ldx + c0 + lane, yo = row * p.ldy + c0 + lane;
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c0 + 32 * k + lane < p.cols ? load_bits<ELEM>(p.x, xo + 32 * k) : 0u;
    if (p.drop.cut) {
      __syncwarp();  // the last part's draws have been read
      *reinterpret_cast<uint4*>(&bits[w][8 * lane]) = drop_bits(key, (uint32_t)(c0 >> 3) + lane, (uint32_t)row);
      __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool keep = p.drop.cut == 0 || bits[w][32 * k + lane] >= p.drop.cut;
      if (c0 + 32 * k + lane < p.cols) store_elem<ELEM>(p.y, yo + 32 * k, keep ? bits_value<ELEM>(v[k]) * p.scale : 0.f);
    }
  }
}

// Rows of 16-byte words: a thread takes groups of eight columns, kItems of them at a time so that their loads are on their
// way together, a whole grid apart; row and group move on by additions.
template <int ELEM>
__global__ void __launch_bounds__(256) dropout_vec_kernel(const DropoutParams p) {
  constexpr int kItems = ELEM == LNFP8_FP32 ? 2 : 4, W = ELEM == LNFP8_FP32 ? 2 : 1, ES = ElemSize<ELEM>::value;
  pdl_wait();
  pdl_launch_dependents();
  drop_save(p.drop);
  const DropKey key = drop_key(p.drop);
  const uint32_t groups = (uint32_t)p.cols >> 3;
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t row = first / groups;
  uint32_t g = (uint32_t)(first - row * groups);
  const uint64_t s2 = pk(p.scale, p.scale);
  while (row < p.rows) {
    int64_t at[kItems];
    uint32_t gr[kItems];
    uint4 u[kItems][W];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      at[i] = row;
      gr[i] = g;
      if (row < p.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + (row * p.ldx + 8 * (int64_t)g) * ES);
#pragma unroll
        for (int k = 0; k < W; ++k) u[i][k] = __ldcs(src + k);
      }
      row += p.step_rows;
      g += p.step_groups;
      if (g >= groups) {
        g -= groups;
        ++row;
      }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (at[i] >= p.rows) break;
      uint64_t v[4];
      unpack8<ELEM>(u[i], v);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = mul_2(v[k], s2);
      if (p.drop.cut) {
        const uint4 d = drop_bits(key, gr[i], (uint32_t)at[i]);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = drop_pair(v[k], w[k], key.cutw);
      }
      uint4 o[W];
      pack8<ELEM>(v, o);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + (at[i] * p.ldy + 8 * (int64_t)gr[i]) * ES);
#pragma unroll
      for (int k = 0; k < W; ++k) __stcs(dst + k, o[k]);
    }
  }
}

template <int ELEM>
lnfp8_status dropout_vec(const DropoutParams& q, cudaStream_t st) {
  constexpr auto kernel = dropout_vec_kernel<ELEM>;
  DropoutParams p = q;
  int bps = 1;
  const lnfp8_status s = kernel_setup<kernel>(256, 0, &bps, "dropout_apply: kernel set-up");
  if (s != LNFP8_OK) return s;
  const int64_t groups = p.cols >> 3;
  const int64_t blocks = min64((p.rows * groups + 255) / 256, (int64_t)num_sms() * bps);
  p.step_rows = blocks * 256 / groups;
  p.step_groups = (uint32_t)(blocks * 256 % groups);
  LaunchScope ls("dropout", st);
  if (launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, st, p) != cudaSuccess) return check_launch("dropout_apply launch");
  return check_launch("dropout_apply");
}

template <int ELEM>
lnfp8_status dropout_any(const DropoutParams& p, cudaStream_t st) {
  const int64_t items = p.rows * ((p.cols + 255) / 256);
  const int64_t blocks = min64((items + kDropWarps - 1) / kDropWarps, (int64_t)num_sms() * 8);
  LaunchScope ls("dropout", st);
  if (launch_pdl(dropout_any_kernel<ELEM>, dim3((unsigned)blocks), dim3(32 * kDropWarps), 0, st, p) != cudaSuccess)
    return check_launch("dropout_apply launch");
  return check_launch("dropout_apply");
}

template <int ELEM>
lnfp8_status dropout(const DropoutParams& p, cudaStream_t st) {
  constexpr int es = ElemSize<ELEM>::value;
  auto rows16 = [](const void* q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * es % 16 == 0; };
  return p.cols % 8 == 0 && rows16(p.x, p.ldx) && rows16(p.y, p.ldy) ? dropout_vec<ELEM>(p, st) : dropout_any<ELEM>(p, st);
}

}  // namespace

lnfp8_status dropout_launch(const void* x, int elem, int64_t rows, int64_t cols, int64_t ldx, const lnfp8_dropout& d, void* y,
                            int64_t ldy, cudaStream_t st) {
  if (rows == 0) return LNFP8_OK;
  DropoutParams p = {};
  p.x = x;
  p.y = y;
  p.rows = rows;
  p.cols = (int)cols;
  p.ldx = ldx;
  p.ldy = ldy;
  p.scale = (float)drop_scale(d);
  p.drop = drop_params(d);
  if (elem == LNFP8_BF16) return dropout<LNFP8_BF16>(p, st);
  return elem == LNFP8_FP16 ? dropout<LNFP8_FP16>(p, st) : dropout<LNFP8_FP32>(p, st);
}

}  // namespace lnfp8
