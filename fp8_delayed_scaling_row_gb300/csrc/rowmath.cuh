// Element types, 8-bit checkpoint blocks and activations shared by the 16/32-bit
// row kernels (layernorm_rows.cu, act_ckpt.cu) and the linear layer (linear.cu).
//
// A checkpoint keeps each 32 consecutive columns of a row as FP8 codes and one
// scale byte b: value = code * 2^(b - 127), with b the least byte for which the
// block's largest magnitude, divided by 2^(b - 127), does not pass the format's
// largest value. The scale is a power of two, so dividing and multiplying by it
// is exact and the code's own rounding (half a step, 2^-4 relative for E4M3,
// 2^-3 for E5M2) is the only one. A block with an Inf or NaN has b = 255 and
// restores as NaN throughout.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace lnfp8 {

template <int ELEM>
struct ElemSize {
  static constexpr int value = ELEM == LNFP8_FP32 ? 4 : 2;
};

template <int ELEM>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (ELEM == LNFP8_FP32) return reinterpret_cast<const float*>(p)[i];
  else if constexpr (ELEM == LNFP8_FP16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
  else return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}

// An element's bits, and their value. Kernels that guard their columns load bits from addresses that are always
// inside and choose afterwards: loads behind a condition would wait for one another.
template <int ELEM>
__device__ __forceinline__ uint32_t load_bits(const void* p, int64_t i) {
  if constexpr (ELEM == LNFP8_FP32) return reinterpret_cast<const uint32_t*>(p)[i];
  else return reinterpret_cast<const uint16_t*>(p)[i];
}
template <int ELEM>
__device__ __forceinline__ float bits_value(uint32_t w) {
  if constexpr (ELEM == LNFP8_FP32) return __uint_as_float(w);
  else if constexpr (ELEM == LNFP8_FP16) return __half2float(__ushort_as_half((unsigned short)w));
  else return __uint_as_float(w << 16);
}

// Parameter vectors (gamma, beta) come in a type of their own, read a few times per block.
__device__ __forceinline__ float load_elem_rt(const void* p, int elem, int64_t i) {
  if (elem == LNFP8_FP32) return load_elem<LNFP8_FP32>(p, i);
  if (elem == LNFP8_FP16) return load_elem<LNFP8_FP16>(p, i);
  return load_elem<LNFP8_BF16>(p, i);
}

template <int ELEM>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
  if constexpr (ELEM == LNFP8_FP32) reinterpret_cast<float*>(p)[i] = v;
  else if constexpr (ELEM == LNFP8_FP16) reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
  else reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// v as it is after being stored in the type (nearest even) and read back.
template <int ELEM>
__device__ __forceinline__ float round_elem(float v) {
  if constexpr (ELEM == LNFP8_FP32) return v;
  else if constexpr (ELEM == LNFP8_FP16) return __half2float(__float2half_rn(v));
  else return __bfloat162float(__float2bfloat16_rn(v));
}

// Packed fp32 pairs: the f32x2 instructions give two IEEE round-to-nearest results each.
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 upk(uint64_t r) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
  return v;
}
__device__ __forceinline__ uint64_t fma_2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub_2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Eight neighbouring elements: one (16-bit types) or two (fp32) 16-byte words.
template <int ELEM>
__device__ __forceinline__ void unpack8(const uint4* u, float* v) {
  if constexpr (ELEM == LNFP8_FP32) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      v[4 * k] = __uint_as_float(u[k].x);
      v[4 * k + 1] = __uint_as_float(u[k].y);
      v[4 * k + 2] = __uint_as_float(u[k].z);
      v[4 * k + 3] = __uint_as_float(u[k].w);
    }
  } else {
    const uint32_t w[4] = {u->x, u->y, u->z, u->w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (ELEM == LNFP8_FP16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
      } else {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    }
  }
}
template <int ELEM>
__device__ __forceinline__ void pack8(const float* v, uint4* u) {
  if constexpr (ELEM == LNFP8_FP32) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      u[k] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (ELEM == LNFP8_FP16) {
        const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
      }
    }
    *u = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// The same as four pairs.
template <int ELEM>
__device__ __forceinline__ void unpack8(const uint4* u, uint64_t* v) {
  float f[8];
  unpack8<ELEM>(u, f);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = pk(f[2 * k], f[2 * k + 1]);
}
template <int ELEM>
__device__ __forceinline__ void pack8(const uint64_t* v, uint4* u) {
  float f[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = upk(v[k]);
    f[2 * k] = t.x;
    f[2 * k + 1] = t.y;
  }
  pack8<ELEM>(f, u);
}
template <int ELEM>
__device__ __forceinline__ void load8(const void* p, int64_t i, float* v) {
  constexpr int W = ELEM == LNFP8_FP32 ? 2 : 1;
  const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p) + i * ElemSize<ELEM>::value);
  uint4 u[W];
#pragma unroll
  for (int k = 0; k < W; ++k) u[k] = q[k];
  unpack8<ELEM>(u, v);
}
__device__ __forceinline__ void load8_rt(const void* p, int elem, int64_t i, float* v) {
  if (elem == LNFP8_FP32) load8<LNFP8_FP32>(p, i, v);
  else if (elem == LNFP8_FP16) load8<LNFP8_FP16>(p, i, v);
  else load8<LNFP8_BF16>(p, i, v);
}
__device__ __forceinline__ void load8_rt(const void* p, int elem, int64_t i, uint64_t* v) {
  float f[8];
  load8_rt(p, elem, i, f);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = pk(f[2 * k], f[2 * k + 1]);
}
template <int ELEM, typename V>  // float[8] or uint64_t[4]
__device__ __forceinline__ void store8(void* p, int64_t i, const V* v) {
  constexpr int W = ELEM == LNFP8_FP32 ? 2 : 1;
  uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p) + i * ElemSize<ELEM>::value);
  uint4 u[W];
  pack8<ELEM>(v, u);
#pragma unroll
  for (int k = 0; k < W; ++k) q[k] = u[k];
}

// One 16-byte word as pairs: 4 of a 16-bit type, 2 of fp32.
template <int ELEM>
__device__ __forceinline__ void unpack_word(const uint4& u, uint64_t* v) {
  if constexpr (ELEM == LNFP8_FP32) {
    v[0] = pk(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = pk(__uint_as_float(u.z), __uint_as_float(u.w));
  } else {
    unpack8<ELEM>(&u, v);
  }
}
template <int ELEM>
__device__ __forceinline__ uint4 pack_word(const uint64_t* v) {
  uint4 u;
  if constexpr (ELEM == LNFP8_FP32) {
    const float2 a = upk(v[0]), b = upk(v[1]);
    u = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  } else {
    pack8<ELEM>(v, &u);
  }
  return u;
}
// The N (4 or 8) parameters from column i on, as pairs.
template <int N>
__device__ __forceinline__ void load_params(const void* p, int elem, int i, uint64_t* v) {
  if constexpr (N == 8) {
    load8_rt(p, elem, i, v);
  } else if (elem == LNFP8_FP32) {
    unpack_word<LNFP8_FP32>(*reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + i), v);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint4 w = make_uint4(u.x, u.y, 0u, 0u);
    uint64_t t[4];
    if (elem == LNFP8_FP16) unpack8<LNFP8_FP16>(&w, t);
    else unpack8<LNFP8_BF16>(&w, t);
    v[0] = t[0];
    v[1] = t[1];
  }
}

// The largest finite value of the type.
template <int ELEM>
__device__ __forceinline__ float elem_max() {
  if constexpr (ELEM == LNFP8_FP32) return __uint_as_float(0x7F7FFFFFu);
  else if constexpr (ELEM == LNFP8_FP16) return 65504.0f;
  else return __uint_as_float(0x7F7F0000u);
}

// 1/sqrt(x) of a variance: the approximation (2 ulp) with one Newton step, within 2 ulp; x = 0
// (a constant row with eps 0) is Inf as by division, x = Inf 0, NaN stays.
__device__ __forceinline__ float rsqrt_nr(float x) {
  const float r = rsqrtf(x);
  const float s = r * fmaf(-0.5f * x * r, r, 1.5f);
  return x > 0.f && x < __uint_as_float(0x7F800000u) ? s : r;
}

// ------------------------------------------------------------ checkpoint blocks
// The scale byte of a block whose largest |v| has these fp32 bits (NaN > Inf > finite):
// the largest value of the format is 1.75 * 2^top, top = 8 (E4M3) or 15 (E5M2).
__device__ __forceinline__ uint32_t ckpt_byte(uint32_t amax_bits, int dt) {
  const int top = dt == LNFP8_E4M3 ? 8 : 15;
  const int e = (int)(amax_bits >> 23);
  if (e == 255) return 255u;
  const int b = e - top + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return b < 0 ? 0u : (uint32_t)b;
}

// 2^(127 - b), the factor of the codes (b <= 247 unless the block is not finite: then NaN).
__device__ __forceinline__ float ckpt_inv_scale(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FFFFFFFu : (254u - b) << 23);
}

// 2^(b - 127); b = 0 is the fp32 subnormal 2^-127, b = 255 NaN.
__device__ __forceinline__ float ckpt_scale(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FFFFFFFu : b << 23);
}

// The codes' format is a run-time argument: it selects one of two conversions, uniformly.
__device__ __forceinline__ uint32_t fp8x2(float a, float b, int dt) {
  return dt == LNFP8_E4M3 ? cvt_fp8x2<LNFP8_E4M3>(a, b) : cvt_fp8x2<LNFP8_E5M2>(a, b);
}
// Eight values times inv -> eight codes.
__device__ __forceinline__ uint2 encode8(const float* v, float inv, int dt) {
  return dt == LNFP8_E4M3 ? cvt_fp8x8<LNFP8_E4M3>(v, inv) : cvt_fp8x8<LNFP8_E5M2>(v, inv);
}
// Two codes (low byte first) -> two fp32, exactly (both formats are subsets of fp16).
__device__ __forceinline__ float2 fp8x2_to_f32(uint32_t codes, int dt) {
  const __half2_raw h = dt == LNFP8_E4M3 ? __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3)
                                         : __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E5M2);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight codes (a uint2, low byte first) times their block's scale.
__device__ __forceinline__ void decode8(uint2 q, float scale, int dt, float* v) {
  const uint32_t w[4] = {q.x & 0xFFFFu, q.x >> 16, q.y & 0xFFFFu, q.y >> 16};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = fp8x2_to_f32(w[k], dt);
    v[2 * k] = f.x * scale;
    v[2 * k + 1] = f.y * scale;
  }
}
__device__ __forceinline__ uint2 encode8(const uint64_t* v, float inv, int dt) {
  const uint64_t i2 = pk(inv, inv);
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = upk(mul_2(v[k], i2));
    c[k] = fp8x2(f.x, f.y, dt);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
// N / 2 pairs times inv -> N codes, low byte first.
template <int N>
__device__ __forceinline__ void encode_pairs(const uint64_t* v, float inv, int dt, uint8_t* dst) {
  if constexpr (N == 8) {
    *reinterpret_cast<uint2*>(dst) = encode8(v, inv, dt);
  } else {
    const uint64_t i2 = pk(inv, inv);
    const float2 a = upk(mul_2(v[0], i2)), b = upk(mul_2(v[1], i2));
    *reinterpret_cast<uint32_t*>(dst) = fp8x2(a.x, a.y, dt) | (fp8x2(b.x, b.y, dt) << 16);
  }
}
__device__ __forceinline__ void decode8(uint2 q, float scale, int dt, uint64_t* v) {
  const uint32_t w[4] = {q.x & 0xFFFFu, q.x >> 16, q.y & 0xFFFFu, q.y >> 16};
  const uint64_t s2 = pk(scale, scale);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = fp8x2_to_f32(w[k], dt);
    v[k] = mul_2(pk(f.x, f.y), s2);
  }
}
// max(|a|, |b|, |c|), NaN if one is (sm_100 and later)
__device__ __forceinline__ float amax3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Largest |v| bits of 8 values, then over the 4 neighbouring lanes that hold a block.
__device__ __forceinline__ uint32_t block_amax8(const float* v) {
  const float m = amax3(amax3(amax3(v[0], v[1], v[2]), v[3], v[4]), amax3(v[5], v[6], v[7]), 0.f);
  uint32_t am = abs_bits(m);
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  return max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
}

__device__ __forceinline__ uint32_t block_amax8(const uint64_t* v) {
  float f[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = upk(v[k]);
    f[2 * k] = t.x;
    f[2 * k + 1] = t.y;
  }
  return block_amax8(f);
}

// The same of 4 values a lane: 8 lanes hold a block.
__device__ __forceinline__ uint32_t block_amax4(const uint64_t* v) {
  const float2 a = upk(v[0]), b = upk(v[1]);
  uint32_t am = abs_bits(amax3(amax3(a.x, a.y, b.x), b.y, 0.f));
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
  return max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 4));
}

// A restored value: code * 2^e, kept inside the type (a block whose largest value
// rounded up past the type's range saturates; NaN stays).
template <int ELEM>
__device__ __forceinline__ float ckpt_clamp(float v) {
  const float m = elem_max<ELEM>();
  return v > m ? m : v < -m ? -m : v;
}

// ------------------------------------------------------------ activations
// GELU is the tanh form, written with the logistic function s(u) = 1/(1 + e^-u):
//   gelu(z) = z s(u), u = 2 sqrt(2/pi) (z + c z^3);  gelu'(z) = s + z s (1 - s) u'
// silu(z) = z s(z); silu'(z) = s + z s (1 - s). ex2.approx and rcp.approx (2 ulp each) and four
// roundings of u log2(e) keep s within (16 + 4 |u|) 2^-24 relative: 2^-20 near 0, 2^-19 at u = -4, 2^-15 at u = -90 (1 + tanh
// would have cancelled long before). That is far below a 16-bit output's half step (2^-8, 2^-11); an fp32 output shows it.
// The .ftz forms: 2^x below 2^-126 is added to 1, and 1/(1 + 2^x) below 2^-126 is a value of no more than
// 128 * 2^-126 lost; the plain forms cost four more instructions each for it.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu2K = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGelu2KC = kGelu2K * 0.044715f;

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// s(u) from -u log2(e)
__device__ __forceinline__ float logistic_neg2(float nu) { return rcp_fast(1.0f + ex2_fast(nu)); }

__device__ __forceinline__ float act_fwd(float z, int act) {
  if (act == LNFP8_ACT_GELU) return z * logistic_neg2(z * (-kLog2e * kGelu2K - kLog2e * kGelu2KC * (z * z)));
  if (act == LNFP8_ACT_SILU) return z * logistic_neg2(-kLog2e * z);
  if (act == LNFP8_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  return z;
}

// relu'(z); a NaN stays one (a lost pre-activation must not pass for an inactive one)
__device__ __forceinline__ float relu_slope(float z) { return z > 0.f ? 1.0f : (z != z ? z : 0.f); }

// act_fwd and the slopes of 8 values as 4 pairs. s(u) of a pair takes one reciprocal, of the product
// (1 + e^-u0)(1 + e^-u1), while the products are in range and none is NaN: kernels that pass over a tensor once are
// bound by the special-function unit otherwise (16 a clock per SM: 2 per value are 58 us for the
// 134 M values of 16384 x 8192, as long as their bytes take).
__device__ __forceinline__ void logistic8(const uint64_t* nu, uint64_t* s) {
  uint64_t d[4];
  float q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 n = upk(nu[k]);
    d[k] = add_2(pk(ex2_fast(n.x), ex2_fast(n.y)), pk(1.0f, 1.0f));
    const float2 t = upk(d[k]);
    q[k] = t.x * t.y;
  }
  // not with a NaN among them, which one reciprocal would carry to the pair's other value (as four comparisons this
  // costs nothing; a maximum that keeps NaN took restore of 16384 x 8192 with GELU from 66 to 72 us)
  if (q[0] < 0x1p120f && q[1] < 0x1p120f && q[2] < 0x1p120f && q[3] < 0x1p120f) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = upk(d[k]);
      const float r = rcp_fast(q[k]);
      s[k] = pk(r * t.y, r * t.x);  // scalar products: a swapped pair would cost moves
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = upk(d[k]);
      s[k] = pk(rcp_fast(t.x), rcp_fast(t.y));
    }
  }
}

// -u log2(e) of GELU's u from z and z^2
__device__ __forceinline__ uint64_t gelu_nu2(uint64_t z, uint64_t zz) {
  return mul_2(z, fma_2(zz, pk(-kLog2e * kGelu2KC, -kLog2e * kGelu2KC), pk(-kLog2e * kGelu2K, -kLog2e * kGelu2K)));
}

template <int ACT>
__device__ __forceinline__ void act8(uint64_t* z) {
  if constexpr (ACT == LNFP8_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = upk(z[k]);
      z[k] = pk(act_fwd(t.x, ACT), act_fwd(t.y, ACT));
    }
  } else if constexpr (ACT != LNFP8_ACT_NONE) {
    uint64_t nu[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      nu[k] = ACT == LNFP8_ACT_GELU ? gelu_nu2(z[k], mul_2(z[k], z[k])) : mul_2(z[k], pk(-kLog2e, -kLog2e));
    logistic8(nu, s);
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = mul_2(z[k], s[k]);
  }
}

// FAR: z may be so large that its square leaves fp32.
template <int ACT, bool FAR>
__device__ __forceinline__ void slope8(const uint64_t* z, uint64_t* out) {
  if constexpr (ACT == LNFP8_ACT_RELU) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = upk(z[k]);
      out[k] = pk(relu_slope(t.x), relu_slope(t.y));
    }
  } else {
    uint64_t nu[4], s[4], zz[4];
    const uint64_t one = pk(1.0f, 1.0f), minus = pk(-1.0f, -1.0f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      zz[k] = mul_2(z[k], z[k]);
      if constexpr (FAR) {
        const float2 t = upk(zz[k]);
        zz[k] = pk(fminf(t.x, 1e30f), fminf(t.y, 1e30f));  // finite, so that the vanished s (1 - s) wins far out
      }
      nu[k] = ACT == LNFP8_ACT_GELU ? gelu_nu2(z[k], zz[k]) : mul_2(z[k], pk(-kLog2e, -kLog2e));
    }
    logistic8(nu, s);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint64_t t = mul_2(mul_2(z[k], s[k]), fma_2(s[k], minus, one));
      if constexpr (ACT == LNFP8_ACT_GELU) {
        const uint64_t du = fma_2(zz[k], pk(3.0f * kGelu2KC, 3.0f * kGelu2KC), pk(kGelu2K, kGelu2K));
        out[k] = fma_2(t, du, s[k]);
      } else {
        out[k] = add_2(t, s[k]);
      }
    }
  }
}

}  // namespace lnfp8
