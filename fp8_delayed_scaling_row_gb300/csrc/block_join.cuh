// The join of a block's output with the residual stream, from one block to the next (a transformer layer around the
// modules of the TE tutorial, code block 2: dropout and residual add behind each sub-layer, a norm in front of the next):
//   forward   n = norm1(x) g1 + b1, h = T(r + s drop(gate n)), y = T(norm2(h) g2 + b2)
//   backward  dH = dh + rs2 (q - [mean(q)] - hhat mean(q hhat)), q = dy g2; dt = s drop'(dH), dn = gate dt,
//             dx = T(rs1 (u - [mean(u)] - xhat mean(u xhat))), u = dn g1; dr = T(dH)
//             ([mean]: layer norms only)
// Each part is optional. All arithmetic is fp32. The forward folds gate, g1 and b1 into one factor and one summand a column,
// gate n = xhat a + c, and s / (1 - p) enters in the sum with r, which then rounds once. (join_fwd_any_kernel folds it into the factor and
// the summand too, or multiplies vector by vector: its h may be the other neighbour of the vector kernel's for the same row.) Of column sums the backward needs four at most, since
// dgate = sum dt n = g1 A + b1 B, dg1 = gate A, db1 = gate B with A = sum dt xhat, B = sum dt.
// This header: what the two kernels of each direction (block_join_fwd.cu, block_join_bwd.cu) share.
#pragma once

#include <initializer_list>

#include "common.cuh"
#include "cp_async.cuh"
#include "internal.h"
#include "kernel_setup.cuh"
#include "philox.cuh"
#include "rowmath.cuh"
#include "rowsum.cuh"

namespace lnfp8 {
namespace {

// A column's parameter, or `none` where there is no such vector.
__device__ __forceinline__ float param_or(const void* p, int elem, int c, float none) { return p ? load_elem_rt(p, elem, c) : none; }

// The parameters of a thread's columns t, t + TPR, ... (tc in place of one it has not, n of them), all on their way together: the
// choice of the type around each load would make it wait for the one before.
template <int ELEM, int TPR, int NE>
__device__ __forceinline__ void load_params_as(const void* p, int tc, int n, float* v) {
  uint32_t b[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) b[i] = load_bits<ELEM>(p, tc + (i < n ? TPR * i : 0));
#pragma unroll
  for (int i = 0; i < NE; ++i) v[i] = bits_value<ELEM>(b[i]);
}
template <int TPR, int NE>
__device__ __forceinline__ void load_params_any(const void* p, int elem, int tc, int n, float* v) {
  if (elem == LNFP8_FP32) load_params_as<LNFP8_FP32, TPR, NE>(p, tc, n, v);
  else if (elem == LNFP8_FP16) load_params_as<LNFP8_FP16, TPR, NE>(p, tc, n, v);
  else load_params_as<LNFP8_BF16, TPR, NE>(p, tc, n, v);
}

// ------------------------------------------------------------ any width, any alignment
// A group of TPR threads owns a row; thread t holds columns t, t + TPR, ..., so that a warp's value i is 32 neighbours:
// four groups of draws. Lane q draws for group q of the warp's NE * 4, and the draws pass through shared memory. A column
// or row that a thread does not have is replaced by one that exists, and its value by zero.
template <int NE>
__device__ __forceinline__ void any_draws(uint16_t* bits, const DropKey& key, int t, int tpr, uint32_t row) {
  const int lane = threadIdx.x & 31, w0 = t & ~31;
  __syncwarp();  // the last row's draws have been read
#pragma unroll
  for (int k = 0; k < NE / 8; ++k) {
    const int q = lane + 32 * k;
    *reinterpret_cast<uint4*>(bits + 8 * q) = drop_bits(key, (uint32_t)(w0 + tpr * (q >> 2)) / 8 + (q & 3), row);
  }
  __syncwarp();
}

// ------------------------------------------------------------ 16-byte rows
// D a multiple of 8 and rows on 16-byte boundaries: thread t of a row's TPR holds its 16-byte words t, t + TPR, ... (EPC
// columns each), 8 to 32 columns in all, and copies (cp.async) the words of its next RING - 1 rows into its own slots of a ring in
// shared memory, so that the bytes in flight cost no registers. Bound by HBM: 16384 x 2048 bf16 with two RMS norms and dropout
// forward 45 us (90% of what a copy of the bytes takes), backward 76 (79%; 71 without dropout). With layer norms, betas and a gate
// 47 and 86 us (85%, 70%): four reductions a row and four column sums, whose registers leave 8 warps an SM.
template <int ELEM>
struct Word {
  static constexpr int EPC = ELEM == LNFP8_FP32 ? 4 : 8;
};

// The draws of a word's columns, two to a register. An fp32 word is half a group of draws. Columns from D on (PART: those of a
// word that the row ends in too) count as dropped: zeros times a row's NaN or infinite sums are NaN, which would be the only ones in a
// row whose own elements are all dropped. (Up to 3% of the time with dropout; zeroed only in such rows, for registers, up to 26%.)
template <int EPC, bool PART = false>
__device__ __forceinline__ void word_draws(const DropKey& key, int c, int D, uint32_t row, uint32_t* w) {
  const uint4 u = drop_bits(key, (uint32_t)c >> 3, row);
  if constexpr (EPC == 8) {
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  } else {
    w[0] = c & 4 ? u.z : u.x;
    w[1] = c & 4 ? u.w : u.y;
  }
#pragma unroll
  for (int k = 0; k < EPC / 2; ++k) {
    if (c + (PART ? 2 * k : 0) >= D) w[k] = 0u;
    else if (PART && c + 2 * k + 1 >= D) w[k] &= 0xFFFFu;
  }
}
// SHIFT: rows of any width on any boundary, the same words of eight columns. A row's aligned words go through the ring (from the
// word that holds its first byte to its last byte, and no further), the group meets before it reads them, and a thread cuts its
// columns out of two neighbours. On the way out a thread joins the last columns of the lane below to its first ones, so that
// all but a warp's and a row's ends leave as aligned words.
__device__ __forceinline__ void shift_words(uint32_t* w, uint32_t bytes) {  // the 16 bytes of 32 from `bytes` < 16 on
#pragma unroll
  for (int k = 0; k < 6; ++k) w[k] = bytes & 8 ? w[k + 2] : w[k];
#pragma unroll
  for (int k = 0; k < 5; ++k) w[k] = bytes & 4 ? w[k + 1] : w[k];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = bytes & 2 ? __funnelshift_r(w[k], w[k + 1], 16) : w[k];
}
__device__ __forceinline__ uint32_t row_shift(const void* p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15); }
// Copies a row's aligned words: thread t words t, t + TPR, ..., and the first the one behind the last.
template <int TPR, int NV>
__device__ __forceinline__ void copy_row(uint32_t dst, const uint8_t* row, int bytes, int t) {
  const uint32_t m = row_shift(row);
  const int end = (int)m + bytes;
  const uint8_t* src = row - m;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int at = (t + TPR * j) * 16;
    if (at < end) cp16_part(dst + at, src + at, min(16, end - at));
  }
  if (t == 0 && TPR * NV * 16 < end) cp16_part(dst + TPR * NV * 16, src + TPR * NV * 16, end - TPR * NV * 16);
}
// Word w (columns c on) of a copied row, zeros from D on.
template <int ELEM>
__device__ __forceinline__ void read_shifted(uint32_t at, uint32_t m, int c, int D, uint64_t* v) {
  constexpr int EPC = Word<ELEM>::EPC;
  const uint4 a = lds16(at), b = lds16(at + 16);
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  shift_words(w, m);
  unpack_word<ELEM>(make_uint4(w[0], w[1], w[2], w[3]), v);
  if (c + EPC > D) {
#pragma unroll
    for (int k = 0; k < EPC / 2; ++k) {
      const float2 f = upk(v[k]);
      v[k] = pk(c + 2 * k < D ? f.x : 0.f, c + 2 * k + 1 < D ? f.y : 0.f);
    }
  }
}
// Writes columns c.. (those below D) of a row; every lane of the warp calls it, `ok` where its row exists.
template <int ELEM, int TPR>
__device__ __forceinline__ void write_shifted(uint8_t* row, int c, int D, int t, bool ok, uint4 u) {
  constexpr int EPC = Word<ELEM>::EPC, ES = ElemSize<ELEM>::value;
  const int lane = threadIdx.x & 31;
  const uint32_t m = row_shift(row);
  uint32_t w[8] = {0u, 0u, 0u, 0u, u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = __shfl_up_sync(0xFFFFFFFFu, w[4 + k], 1);
  // the aligned word that this thread's first columns end: m bytes of the lane below, then its own
  const int head = (int)(16 - m) / ES;
  const bool full = ok && c + head <= D && (m == 0 || (lane > 0 && t > 0));
  const bool above = __shfl_down_sync(0xFFFFFFFFu, (int)full, 1) && lane < 31 && t < TPR - 1;  // takes the rest
  if (m != 0) shift_words(w, 16 - m);
  else
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = w[k + 4];
  if (full) *reinterpret_cast<uint4*>(row - m + (int64_t)c * ES) = make_uint4(w[0], w[1], w[2], w[3]);
  if (!ok) return;
  const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < EPC; ++k) {
    if (c + k >= D || (k < head ? full : above)) continue;
    if constexpr (ELEM == LNFP8_FP32) reinterpret_cast<uint32_t*>(row)[c + k] = e[k];
    else reinterpret_cast<uint16_t*>(row)[c + k] = (uint16_t)(e[k / 2] >> (16 * (k & 1)));
  }
}
template <int TPR>
__device__ __forceinline__ void group_meet() {
  if constexpr (TPR <= 32) __syncwarp();
  else group_sync<TPR>();
}

// One block to an SM, of 512 threads (backward 256, 384 or 512: bwd_threads), whose row groups share the columns' factors: in fp32
// in shared memory, 16 bytes of neighbouring lanes side by side, ready to be used (in registers they cost a block's worth of
// occupancy, read again as parameters 60 instructions a row). FULL: with means (layer norms) and betas; without them (RMS) rows cost
// half the instructions. Rows on odd boundaries always run as FULL.
constexpr int kVecThreads = 512;
constexpr int kVecSmem = 226 * 1024;

// Four columns of a factor array: quarter q of the row's words' quarters.
template <int T, int TPR, int NV, int EPC>
__device__ __forceinline__ void put_factors(uint4* at, int k, const void* a, const void* b, int elem, float scale, float none, int D) {
  constexpr int Q = NV * EPC / 4;  // of a thread
  float4* dst = reinterpret_cast<float4*>(at) + k * Q * TPR;
  for (int i = threadIdx.x; i < Q * TPR; i += T) {
    const int t = i % TPR, q = i / TPR, c = (t + TPR * (q * 4 / EPC)) * EPC + q * 4 % EPC;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c + e < D ? scale * param_or(a, elem, c + e, none) * param_or(b, elem, c + e, 1.f) : 0.f;
    dst[i] = make_float4(v[0], v[1], v[2], v[3]);
  }
}
// A word's parameters as pairs, `none` where there is no such vector.
template <int EPC>
__device__ __forceinline__ void params_or(const void* p, int elem, int c, float none, uint64_t* v) {
  if (p) {
    load_params<EPC>(p, elem, c, v);
  } else {
#pragma unroll
    for (int k = 0; k < EPC / 2; ++k) v[k] = pk(none, none);
  }
}
template <int TPR, int NV, int EPC>
__device__ __forceinline__ void get_factors(uint32_t at, int k, int j, uint64_t* v) {
  constexpr int Q = NV * EPC / 4;
#pragma unroll
  for (int h = 0; h < EPC / 4; ++h) {
    const uint4 u = lds16(at + ((k * Q + j * (EPC / 4) + h) * TPR) * 16);
    v[2 * h] = pk(__uint_as_float(u.x), __uint_as_float(u.y));
    v[2 * h + 1] = pk(__uint_as_float(u.z), __uint_as_float(u.w));
  }
}

inline bool vectors_aligned(std::initializer_list<const void*> v) {
  for (const void* p : v)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}
inline bool row_aligned(const void* p, int64_t ld, int es) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0; }

}  // namespace
}  // namespace lnfp8
