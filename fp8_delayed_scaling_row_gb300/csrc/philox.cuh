// The draws of dropout: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011), a bijection of a 128-bit counter under a 64-bit key. A mask is a function of its place, so nothing is stored
// and the backward draws the same again.
//   key      seed, low word first
//   counter  (column / 8, row, step, site)
// The eight 16-bit parts of the four words belong to eight neighbouring columns, low part first. 16 bits take p to
// 2^-16, and one call serves eight elements: ten rounds are about 60 instructions, 7.5 an element, where the bytes of a
// 16-bit element take an SM 0.35 clocks of its 128 lanes, 44 instructions' time.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace lnfp8 {

// What a kernel gets of an lnfp8_dropout.
struct DropParams {
  const int64_t* rng;
  int64_t* rng_saved;
  uint32_t cut, site;  // dropped below `cut`, 0: nothing is drawn
};

inline DropParams drop_params(const lnfp8_dropout& d) {
  DropParams p;
  p.rng = d.rng;
  p.rng_saved = d.rng ? d.rng_saved : nullptr;
  p.cut = drop_threshold(d.p);
  p.site = d.site;
  return p;
}
// What is kept is divided by the probability of being kept (nothing is with cut = 65536).
inline double drop_scale(const lnfp8_dropout& d) {
  const uint32_t cut = drop_threshold(d.p);
  return cut >= 65536 ? 0.0 : 65536.0 / (65536.0 - cut);
}

// `cut` as the high half of a word to compare draws with. Where everything is dropped (cut 65536) draws are zeros
// instead, below any other cut.
struct DropKey {
  uint32_t k0, k1, step, site, cutw;
  bool all;
};
__device__ __forceinline__ DropKey drop_key(const DropParams& d) {
  DropKey k = {0u, 0u, 0u, d.site, d.cut > 65535u ? 0xFFFF0000u : d.cut << 16, d.cut > 65535u};
  if (d.cut) {
    const uint64_t seed = (uint64_t)d.rng[0];
    k.k0 = (uint32_t)seed;
    k.k1 = (uint32_t)(seed >> 32);
    k.step = (uint32_t)d.rng[1];
  }
  return k;
}
// One thread of the grid keeps the backward's copy.
__device__ __forceinline__ void drop_save(const DropParams& d) {
  if (d.rng_saved && blockIdx.x == 0 && threadIdx.x == 0) {
    d.rng_saved[0] = d.rng[0];
    d.rng_saved[1] = d.rng[1];
  }
}

// The draws of columns 8 group .. 8 group + 7 of a row.
__device__ __forceinline__ uint4 drop_bits(const DropKey& key, uint32_t group, uint32_t row) {
  uint32_t c0 = group, c1 = row, c2 = key.step, c3 = key.site, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return key.all ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(c0, c1, c2, c3);
}

// Two neighbouring elements, zero where their draws (the halves of w) are below the cut.
__device__ __forceinline__ uint64_t drop_pair(uint64_t v, uint32_t w, uint32_t cutw) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  lo = (w << 16) >= cutw ? lo : 0.f;
  hi = w >= cutw ? hi : 0.f;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}

}  // namespace lnfp8
