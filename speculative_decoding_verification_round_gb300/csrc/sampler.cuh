// sampler.cuh -- the sampler's arithmetic, shared by the acceptance of drafts
// (accept.cu) and the filtered sampling (sample.cu): the fp32 exp and integer
// weights, order keys of logits, exact thresholds.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace {

typedef unsigned __int128 u128;

// ---------------------------------------------------------------------------
// the sampler's exp and integer weight (fp32, no contraction: __f*_rn)
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t int_weight(float x) {
  if (!(x >= -87.0f)) return 0ull;
  const float LOG2E = 0x1.715476p+0f;     // fl32(1 / ln 2)
  const float LN2_HI = 0x1.62e4p-1f;      // ln 2 to 12 significant bits
  const float LN2_LO = 0x1.7f7d1cp-20f;   // fl32(ln 2 - LN2_HI)
  const float C[8] = {0x1p+0f,        0x1p+0f,        0x1p-1f,         0x1.555556p-3f,
                      0x1.555556p-5f, 0x1.111112p-7f, 0x1.6c16c2p-10f, 0x1.a01a02p-13f};
  const float n = rintf(__fmul_rn(x, LOG2E));
  float r = __fsub_rn(x, __fmul_rn(n, LN2_HI));
  r = __fsub_rn(r, __fmul_rn(n, LN2_LO));
  float p = C[7];
#pragma unroll
  for (int k = 6; k >= 0; k--) p = __fadd_rn(__fmul_rn(p, r), C[k]);
  const int e = (int)n + 32;
  if (e < 0) return 0ull;
  const float v = __fmul_rn(p, __int_as_float((e + 127) << 23));
  return (uint64_t)v;  // truncation: exact floor of a non-negative value
}

// floor(U * total / 2^32) without overflowing 128 bits
__device__ __forceinline__ u128 scaled_threshold(uint32_t U, u128 total) {
  const u128 hi = total >> 32, lo = total & 0xFFFFFFFFull;
  return (u128)U * hi + (((u128)U * lo) >> 32);
}

// Order-preserving 32-bit key of a float (-0 taken as +0).  Keys of the
// same row are only compared and turned back into the value.
__device__ __forceinline__ uint32_t max_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// The row's max z from the key of its largest logit.
__device__ __forceinline__ float row_zmax(uint32_t key, float T) {
  const float m = key_value(key);
  return T == 1.0f ? m : __fdiv_rn(m, T);
}
__device__ __forceinline__ float zval(float l, float T) {
  return T == 1.0f ? l : __fdiv_rn(l, T);  // x / 1 is x exactly
}

}  // namespace
