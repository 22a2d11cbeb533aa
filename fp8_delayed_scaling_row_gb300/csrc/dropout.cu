// Dropout whose mask is never stored: y = x / (1 - p) where the element's draw keeps it, else 0. The backward is the
// same map on the gradient. Bound by HBM: an element is read once and written once.
#include "common.cuh"
#include "internal.h"
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

template <int ELEM>
lnfp8_status dropout_any(const DropoutParams& p, cudaStream_t st) {
  const int64_t items = p.rows * ((p.cols + 255) / 256);
  const int64_t blocks = min64((items + kDropWarps - 1) / kDropWarps, (int64_t)num_sms() * 8);
  LaunchScope ls("dropout", st);
  if (launch_pdl(dropout_any_kernel<ELEM>, dim3((unsigned)blocks), dim3(32 * kDropWarps), 0, st, p) != cudaSuccess)
    return check_launch("dropout_apply launch");
  return check_launch("dropout_apply");
}

}  // namespace

lnfp8_status dropout_launch(const void* x, int elem, int64_t rows, int64_t cols, int64_t ldx, const lnfp8_dropout& d, void* y,
                            int64_t ldy, cudaStream_t st) {
  if (rows == 0) return LNFP8_OK;
  DropoutParams p;
  p.x = x;
  p.y = y;
  p.rows = rows;
  p.cols = (int)cols;
  p.ldx = ldx;
  p.ldy = ldy;
  p.scale = (float)drop_scale(d);
  p.drop = drop_params(d);
  if (elem == LNFP8_BF16) return dropout_any<LNFP8_BF16>(p, st);
  return elem == LNFP8_FP16 ? dropout_any<LNFP8_FP16>(p, st) : dropout_any<LNFP8_FP32>(p, st);
}

}  // namespace lnfp8
