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

// Any width and alignment, bound by its accesses of one element (16384 x 8191 bf16 153 us, fp32 8192 x 8191 93): a warp takes
// 256 columns of a row. Lane q draws for the q-th group of eight, and the draws go through shared memory to the lanes that hold
// the columns (32 neighbours at a time).
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

// The same of rows of up to 128 columns, where a warp a row would leave most of its draws unused: a warp takes 32 groups of eight
// columns one after another, from one row into the next, and the lane of a column gets its row and group from the lane that
// drew for it.
template <int ELEM>
__global__ void __launch_bounds__(32 * kDropWarps) dropout_narrow_kernel(const DropoutParams p) {
  __shared__ __align__(16) uint16_t bits[kDropWarps][256];
  pdl_wait();
  pdl_launch_dependents();
  drop_save(p.drop);
  const DropKey key = drop_key(p.drop);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t groups = ((uint32_t)p.cols + 7) >> 3;
  const int64_t items = p.rows * groups;
  for (int64_t i0 = ((int64_t)blockIdx.x * kDropWarps + w) * 32; i0 < items; i0 += (int64_t)gridDim.x * kDropWarps * 32) {
    const int64_t item = i0 + lane;
    const bool in = item < items;
    const uint32_t row = in ? (uint32_t)(item / groups) : 0u, g = in ? (uint32_t)(item - (int64_t)row * groups) : groups;  // past every column
    uint32_t v[8], r[8], c[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      r[k] = __shfl_sync(0xFFFFFFFFu, row, 4 * k + (lane >> 3));
      c[k] = 8 * __shfl_sync(0xFFFFFFFFu, g, 4 * k + (lane >> 3)) + (lane & 7);
      v[k] = c[k] < (uint32_t)p.cols ? load_bits<ELEM>(p.x, (int64_t)r[k] * p.ldx + c[k]) : 0u;
    }
    if (p.drop.cut) {
      __syncwarp();  // the last draws have been read
      *reinterpret_cast<uint4*>(&bits[w][8 * lane]) = drop_bits(key, g, row);
      __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool keep = p.drop.cut == 0 || bits[w][32 * k + lane] >= key.cutw >> 16;
      if (c[k] < (uint32_t)p.cols) store_elem<ELEM>(p.y, (int64_t)r[k] * p.ldy + c[k], keep ? bits_value<ELEM>(v[k]) * p.scale : 0.f);
    }
  }
}

// Rows of whole groups of eight columns, one access of 16 or (fp32) 32 bytes each: a thread takes kItems of them at a time, so
// that their loads are on their way together, a whole grid apart; row and group move on by additions. 16384 x 8192 bf16 95 us (two
// items 100, eight 113, with streaming accesses 99), 84% of a copy: 2.2 of an SM's 4 instructions a clock, the wide
// multiplications' pipe at 64%. 8192 x 8192 fp32 88 us, 91% (as two 16-byte accesses 110).
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
        const uint8_t* src = static_cast<const uint8_t*>(p.x) + (row * p.ldx + 8 * (int64_t)g) * ES;
        if constexpr (W == 1) u[i][0] = *reinterpret_cast<const uint4*>(src);
        else load32(src, reinterpret_cast<uint32_t*>(u[i]));
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
      uint8_t* dst = static_cast<uint8_t*>(p.y) + (at[i] * p.ldy + 8 * (int64_t)gr[i]) * ES;
      if constexpr (W == 1) *reinterpret_cast<uint4*>(dst) = o[0];
      else store32(dst, reinterpret_cast<const uint32_t*>(o));
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
  const bool narrow = p.cols <= 128;
  const int64_t items = narrow ? (p.rows * ((p.cols + 7) / 8) + 31) / 32 : p.rows * ((p.cols + 255) / 256);
  const int64_t blocks = min64((items + kDropWarps - 1) / kDropWarps, (int64_t)num_sms() * 8);
  LaunchScope ls("dropout", st);
  if (launch_pdl(narrow ? dropout_narrow_kernel<ELEM> : dropout_any_kernel<ELEM>, dim3((unsigned)blocks), dim3(32 * kDropWarps), 0, st, p) != cudaSuccess)
    return check_launch("dropout_apply launch");
  return check_launch("dropout_apply");
}

template <int ELEM>
lnfp8_status dropout(const DropoutParams& p, cudaStream_t st) {
  constexpr int es = ElemSize<ELEM>::value;
  // a group of eight columns is one access, of 16 or 32 bytes
  auto whole = [](const void* q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % (8 * es) == 0 && ld % 8 == 0; };
  return p.cols % 8 == 0 && whole(p.x, p.ldx) && whole(p.y, p.ldy) ? dropout_vec<ELEM>(p, st) : dropout_any<ELEM>(p, st);
}

}  // namespace

lnfp8_status drop_save_launch(const lnfp8_dropout& d, const char* who, cudaStream_t st) {
  if (!d.rng || !d.rng_saved) return LNFP8_OK;
  if (cudaMemcpyAsync(d.rng_saved, d.rng, 2 * sizeof(int64_t), cudaMemcpyDeviceToDevice, st) != cudaSuccess) return check_launch(who);
  return LNFP8_OK;
}

lnfp8_status dropout_launch(const void* x, int elem, int64_t rows, int64_t cols, int64_t ldx, const lnfp8_dropout& d, void* y,
                            int64_t ldy, cudaStream_t st) {
  if (rows == 0) return drop_save_launch(d, "dropout_apply", st);
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
