// key_warp.cuh -- one warp's attention of 8 NT query rows to keys in shared
// memory, 16 at a time, with mma.sync: rows of fp16 or of 4-bit codes.  Internal.
//
// The keys are the M of the products and the query rows the N, S^T = K Q^T and
// O^T += V^T P^T, so that the few rows of a decode step (a GQA group, 4 to 8)
// fill a tile of 8 instead of half of one of 16.  What the layout of the
// fragments asks of K, V and Q is met by choosing the order of the dimensions
// and keys, which no sum depends on:
//   4-bit K  lane (g, t) takes the word t of each block of 32 elements of its keys: a
//            nibble by itself is a (subnormal) fp16 number, u 2^-24 or, four bits
//            higher, u 2^-20, so that four masks and a shift give eight elements of the
//            operand.  Both kinds have a sum of their own; u = q + 8: the first one
//            starts at -8 2^-24 sum q of the block, and the block's scale multiplies
//            them in fp32.
//   4-bit V  ldmatrix turns 16 bits, four elements, of eight keys to pairs of keys:
//            lane (g, t) has elements 2g, 2g + 1, 16 + 2g, 17 + 2g of each block of keys 2t, 2t + 1.
//            The number 1024 + u by its bits, minus 1032, times the pair's scales, both
//            exact in fp16 (a scale has eight significant bits, u - 8 three).
// A row's elements so belong to the accumulator tiles in another order than in
// fp16 (dim_of).
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace {

// The running maximum lags behind by up to 2^KW_SLACK, which saves the
// reductions over the lanes, and 2^KW_BIAS multiplies weights and sums, which
// keeps what lies far below the maximum inside fp16's range: a pair of fp16
// numbers holds all of a weight w but 2^-20 w + 2^-36.
constexpr float KW_SLACK = 3.0f, KW_BIAS = 12.0f;
// hi is the weight cut off behind its 11th bit, lo the rest and 2^-22 of hi
// more: both are non-negative, and an infinite value stays infinite.
constexpr uint32_t KW_CUT = 0xFFFFE000u;
constexpr float KW_REST = 1.0f - 0x1p-22f;

__device__ __forceinline__ uint32_t kw_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t kw_lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t kw_lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 kw_lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint4 kw_lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void kw_sts64(uint32_t at, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void kw_sts128f(uint32_t at, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
// BYTES to shared memory; zeros if !valid (src is then any readable address).
template <int BYTES>
__device__ __forceinline__ void kw_copy(uint32_t dst, const void* src, bool valid) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(valid ? BYTES : 0));
}
__device__ __forceinline__ uint32_t kw_pack(float a, float b) {  // a in the low half
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float kw_half(uint32_t v, int hi) {
  return __half2float(__ushort_as_half((unsigned short)(hi ? v >> 16 : v & 0xFFFFu)));
}
__device__ __forceinline__ float kw_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two floats at a time: x y + z, x + y.
__device__ __forceinline__ void kw_fma2(float& r0, float& r1, float x0, float x1, float y0, float y1, float z0, float z1) {
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r0), "=f"(r1) : "f"(x0), "f"(x1), "f"(y0), "f"(y1), "f"(z0), "f"(z1));
}
__device__ __forceinline__ void kw_mul2(float& r0, float& r1, float x0, float x1, float y0, float y1) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r0), "=f"(r1) : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
}
__device__ __forceinline__ void kw_add2(float& r0, float& r1, float x0, float x1, float y0, float y1) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r0), "=f"(r1) : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
}
__device__ __forceinline__ uint32_t kw_transpose(uint32_t v) {  // 8 x 8 of 16 bits
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t kw_hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t kw_hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t kw_hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// u - 8 of two nibbles: those at bits 0-3 and 16-19, and those at bits 4-7 and 20-23.
__device__ __forceinline__ uint32_t q4_low(uint32_t x) {  // (1024 + u) - 1032
  return kw_hadd2(lop3_and_or(x, 0x000F000Fu, 0x64006400u), 0xE408E408u);
}
__device__ __forceinline__ uint32_t q4_high(uint32_t x) {  // (1024 + 16 u) / 16 - 72
  return kw_hfma2(lop3_and_or(x, 0x00F000F0u, 0x64006400u), 0x2C002C00u, 0xD480D480u);
}
__device__ __forceinline__ bool odd_half(uint32_t v) { return (v & 0x7C00u) == 0x7C00u; }  // infinite or NaN
// A scale that makes infinities or NaN of codes: one itself, or 8192 and more, 8 times which fp16 does not hold.
__device__ __forceinline__ bool odd_scale(uint32_t v) { return (v & 0x7FFFu) >= 0x7000u; }
__device__ __forceinline__ bool odd_pair(uint32_t v) { return odd_half(v) || odd_half(v >> 16); }

// What code u stands for: the product rounded to fp16, as kw_hmul2 makes it.
__device__ __forceinline__ float q4_value(int u, float scale) {
  return __half2float(__float2half_rn((float)(u - 8) * scale));
}

// A row of codes: HD / 2 bytes, 16-byte chunk c of row r at c ^ q4_swz(r), so that a chunk
// of eight rows, read as words or by ldmatrix, lies in all banks.
template <int HD>
__device__ __forceinline__ int q4_swz(int r) {
  return HD == 128 ? r >> 1 & 3 : r >> 2 & 1;
}
// A row of fp16: HD * 2 bytes, 16-byte unit u of row r at u ^ (r & 7).
template <int HD>
__device__ __forceinline__ uint32_t f16_off(int r, int u) {
  return (uint32_t)(r * (HD * 2) + ((u ^ (r & 7)) << 4));
}

// Q4: the order of the dimensions that the codes ask for.
template <int HD, int NT, bool Q4>
struct KeyWarp {
  static constexpr int STEPS = HD / 16, BLOCKS = HD / 32, MTILES = HD / 16;
  static constexpr int Q_BYTES = STEPS * NT * 32 * 8;     // query fragments of a CTA
  static constexpr int SUM_BYTES = BLOCKS * NT * 4 * 16;  // and sums of their blocks (Q4), as accumulators begin
  int g, t;
  float o[MTILES][NT][4];  // (dimension g of a tile; rows 2t, 2t + 1), (dimension g + 8; ...)
  float mx[NT][2], sum[NT][2];  // of rows 2t, 2t + 1; sum: this lane's keys

  __device__ __forceinline__ void begin() {
    g = (threadIdx.x & 31) >> 2;
    t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
      for (int m = 0; m < MTILES; m++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[m][n][e] = 0.0f;
      mx[n][0] = mx[n][1] = -INFINITY;
      sum[n][0] = sum[n][1] = 0.0f;
    }
  }

  // The dimension of accumulator tile m's row `half` (0: g, 1: g + 8).
  __device__ __forceinline__ int dim_of(int m, int half) const {
    return Q4 ? 32 * (m >> 1) + 16 * half + 2 * g + (m & 1) : 16 * m + 8 * half + g;
  }

  // Query fragments: entry e of (step, n, lane), row(r): row r's data or null.
  // Every thread of the CTA; `threads` of them.  neg: the scores' scale is negative,
  // which the queries take over, so that a row's largest score has its largest product.
  template <class F>
  static __device__ __forceinline__ void put_queries(uint32_t qs, uint32_t sums, int tid, int threads, bool neg, F&& row) {
    const uint32_t sign = neg ? 0x80008000u : 0u;
    for (int e = tid; e < STEPS * NT * 32; e += threads) {
      const int lane = e & 31, n = e / 32 % NT, step = e / 32 / NT;
      const __half* p = row(8 * n + (lane >> 2));
      uint32_t b0 = 0u, b1 = 0u;
      if (p != nullptr) {
        if (Q4) {  // elements 4t, 4t + 2 and 4t + 1, 4t + 3
          const uint2 v = *reinterpret_cast<const uint2*>(p + 16 * step + 4 * (lane & 3));
          b0 = __byte_perm(v.x, v.y, 0x5410);
          b1 = __byte_perm(v.x, v.y, 0x7632);
        } else {
          b0 = *reinterpret_cast<const uint32_t*>(p + 16 * step + 2 * (lane & 3));
          b1 = *reinterpret_cast<const uint32_t*>(p + 16 * step + 2 * (lane & 3) + 8);
        }
      }
      kw_sts64(qs + e * 8, b0 ^ sign, b1 ^ sign);
    }
    if (Q4)
      for (int e = tid; e < BLOCKS * NT * 4; e += threads) {
        const int tt = e & 3, n = e / 4 % NT, b = e / 4 / NT;
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const __half* p = row(8 * n + 2 * tt + h);
          if (p != nullptr)
#pragma unroll
            for (int u = 0; u < 4; u++) {
              const uint4 v = *reinterpret_cast<const uint4*>(p + 32 * b + 8 * u);
              s[h] += kw_half(v.x, 0) + kw_half(v.x, 1) + kw_half(v.y, 0) + kw_half(v.y, 1) + kw_half(v.z, 0) +
                      kw_half(v.z, 1) + kw_half(v.w, 0) + kw_half(v.w, 1);
            }
        }
        const float f = neg ? 0x1p-21f : -0x1p-21f;
        kw_sts128f(sums + e * 16, s[0] * f, s[1] * f, s[0] * f, s[1] * f);
      }
  }

  // x = 2^-24 K Q^T of KT tiles of 16 rows of codes at `ks` (their scales at `ss`).
  // Lane (g, t): keys g and g + 8 of each tile, rows 2t, 2t + 1 of each n.
  template <int KT>
  __device__ __forceinline__ void scores_q4(uint32_t ks, uint32_t ss, uint32_t qs, uint32_t sums,
                                            float (&x)[KT][NT][4]) const {
    const int lane = g * 4 + t;
    const uint32_t k0 = ks + g * (HD / 2) + 4 * t + (q4_swz<HD>(g) << 4), s0 = ss + g * (HD / 16);
    uint32_t sc[KT][2][BLOCKS / 2];
#pragma unroll
    for (int i = 0; i < KT; i++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const uint32_t at = s0 + (16 * i + 8 * h) * (HD / 16);
        if (BLOCKS == 4) {
          const uint2 v = kw_lds64(at);
          sc[i][h][0] = v.x;
          sc[i][h][BLOCKS / 2 - 1] = v.y;
        } else {
          sc[i][h][0] = kw_lds32(at);
        }
      }
#pragma unroll
    for (int b = 0; b < BLOCKS; b++) {
      uint32_t w[KT][2];
      const uint32_t kb = k0 ^ (b << 4);
#pragma unroll
      for (int i = 0; i < KT; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) w[i][h] = kw_lds32(kb + (16 * i + 8 * h) * (HD / 2));
      float low[KT][NT][4], high[KT][NT][4];  // of elements 0-15 and of 16-31, these 16 times
      uint32_t al[KT][4], ah[KT][4];
#pragma unroll
      for (int i = 0; i < KT; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t v = w[i][h] >> 8;
          al[i][h] = w[i][h] & 0x000F000Fu;
          al[i][2 + h] = v & 0x000F000Fu;
          ah[i][h] = w[i][h] & 0x00F000F0u;
          ah[i][2 + h] = v & 0x00F000F0u;
        }
#pragma unroll
      for (int n = 0; n < NT; n++) {
        const uint2 ql = kw_lds64(qs + ((2 * b * NT + n) * 32 + lane) * 8);
        const uint2 qh = kw_lds64(qs + (((2 * b + 1) * NT + n) * 32 + lane) * 8);
        const uint4 cc = kw_lds128(sums + ((b * NT + n) * 4 + t) * 16);
        const float c[4] = {__uint_as_float(cc.x), __uint_as_float(cc.y), __uint_as_float(cc.z), __uint_as_float(cc.w)};
#pragma unroll
        for (int i = 0; i < KT; i++) {
          mma_16816_c(low[i][n], al[i], ql.x, ql.y, c);
          mma_16816_zero(high[i][n], ah[i], qh.x, qh.y);
        }
      }
#pragma unroll
      for (int i = 0; i < KT; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const float s = kw_half(sc[i][h][b >> 1], b & 1);
#pragma unroll
          for (int n = 0; n < NT; n++) {
            float* y = &x[i][n][2 * h];
            const float* l = &low[i][n][2 * h];
            const float* u = &high[i][n][2 * h];
            float z0, z1;
            kw_fma2(z0, z1, u[0], u[1], 0.0625f, 0.0625f, l[0], l[1]);
            if (b == 0)
              kw_mul2(y[0], y[1], z0, z1, s, s);
            else
              kw_fma2(y[0], y[1], z0, z1, s, s, y[0], y[1]);
          }
        }
    }
  }
  static constexpr float CODE_UNIT = 0x1p24f;  // of these scores

  // K Q^T of one tile of 16 fp16 rows.
  __device__ __forceinline__ void scores_f16(uint32_t ks, uint32_t qs, float (&x)[NT][4]) const {
    const int lane = g * 4 + t;
#pragma unroll
    for (int step = 0; step < STEPS; step++) {
      uint32_t a[4];
      if (Q4) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int r = 8 * h + g;
          const uint2 v = kw_lds64(ks + f16_off<HD>(r, 2 * step + (t >> 1)) + 8 * (t & 1));
          a[h] = __byte_perm(v.x, v.y, 0x5410);
          a[2 + h] = __byte_perm(v.x, v.y, 0x7632);
        }
      } else {
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                     : "r"(ks + f16_off<HD>(lane & 15, 2 * step + (lane >> 4))));
      }
#pragma unroll
      for (int n = 0; n < NT; n++) {
        const uint2 q = kw_lds64(qs + ((step * NT + n) * 32 + lane) * 8);
        if (step == 0)
          mma_16816_zero(x[n], a, q.x, q.y);
        else
          mma_16816(x[n], a, q.x, q.y);
      }
    }
  }

  // Scores x, f > 0 times which are in log2 units, to weights (times 2^KW_BIAS); the
  // running maximum and sum.
  template <int KT>
  __device__ __forceinline__ void weights(float f, float (&x)[KT][NT][4]) {
    bool grow = false;
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        top[n][h] = fmaxf(x[0][n][h], x[0][n][2 + h]);
#pragma unroll
        for (int i = 1; i < KT; i++) top[n][h] = fmaxf(top[n][h], fmaxf(x[i][n][h], x[i][n][2 + h]));
        top[n][h] *= f;
        grow |= top[n][h] > mx[n][h] + KW_SLACK;  // (-infinity + 3 at first)
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NT; n++) {
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float m = fmaxf(mx[n][h], top[n][h]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
          al[h] = m == -INFINITY ? 1.0f : kw_exp2(mx[n][h] - m);
          mx[n][h] = m;
          sum[n][h] *= al[h];
        }
#pragma unroll
        for (int m = 0; m < MTILES; m++)
#pragma unroll
          for (int e = 0; e < 4; e++) o[m][n][e] *= al[e & 1];
      }
    }
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const float s0 = KW_BIAS - (mx[n][0] == -INFINITY ? 0.0f : mx[n][0]);
      const float s1 = KW_BIAS - (mx[n][1] == -INFINITY ? 0.0f : mx[n][1]);
#pragma unroll
      for (int i = 0; i < KT; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float* y = &x[i][n][2 * h];
          kw_fma2(y[0], y[1], y[0], y[1], f, f, s0, s1);
          y[0] = kw_exp2(y[0]);
          y[1] = kw_exp2(y[1]);
          kw_add2(sum[n][0], sum[n][1], sum[n][0], sum[n][1], y[0], y[1]);
        }
    }
  }

  // A tile's weights as fragments: pairs of fp16 numbers hi + lo.
  __device__ __forceinline__ void split(const float (&p)[NT][4], uint32_t (&hi)[NT][2], uint32_t (&lo)[NT][2]) const {
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const float a = p[n][2 * h], b = p[n][2 * h + 1];
        const float ca = __uint_as_float(__float_as_uint(a) & KW_CUT), cb = __uint_as_float(__float_as_uint(b) & KW_CUT);
        float ra, rb;
        kw_fma2(ra, rb, ca, cb, -KW_REST, -KW_REST, a, b);
        hi[n][h] = kw_transpose(kw_pack(ca, cb));
        lo[n][h] = kw_transpose(kw_pack(ra, rb));
      }
  }
  __device__ __forceinline__ void add(int m, const uint32_t (&a)[4], const uint32_t (&hi)[NT][2],
                                      const uint32_t (&lo)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; n++) {
      mma_16816(o[m][n], a, hi[n][0], hi[n][1]);
      mma_16816(o[m][n], a, lo[n][0], lo[n][1]);
    }
  }

  // O += P V of one tile of 16 rows of codes at `vs`, scales at `ss`.
  __device__ __forceinline__ void values_q4(uint32_t vs, uint32_t ss, const float (&p)[NT][4]) {
    uint32_t hi[NT][2], lo[NT][2];
    split(p, hi, lo);
    // the scales of keys 2t, 2t + 1 | 2t + 8, 2t + 9 of each block
    uint32_t s[BLOCKS][2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t at = ss + (2 * t + 8 * h) * (HD / 16);
      uint32_t a[2], b[2];
      if (HD == 128) {
        const uint4 v = kw_lds128(at);  // both keys'
        a[0] = v.x, a[1] = v.y, b[0] = v.z, b[1] = v.w;
      } else {
        const uint2 v = kw_lds64(at);
        a[0] = v.x, b[0] = v.y;
      }
#pragma unroll
      for (int x = 0; x < BLOCKS; x++) s[x][h] = __byte_perm(a[x >> 1], b[x >> 1], x & 1 ? 0x7632 : 0x5410);
    }
    const int lane = g * 4 + t, key = lane & 15;
    const uint32_t v0 = vs + key * (HD / 2) + (((lane >> 4) ^ q4_swz<HD>(key)) << 4);
#pragma unroll
    for (int c = 0; c < BLOCKS; c += 2) {
      uint32_t w[4];  // blocks c, c + 1 of keys 0-7 and 8-15
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(v0 ^ (c << 4)));
#pragma unroll
      for (int b = 0; b < 2; b++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const uint32_t x0 = j ? w[2 * b] >> 8 : w[2 * b], x1 = j ? w[2 * b + 1] >> 8 : w[2 * b + 1];
          const uint32_t a[4] = {kw_hmul2(q4_low(x0), s[c + b][0]), kw_hmul2(q4_high(x0), s[c + b][0]),
                                 kw_hmul2(q4_low(x1), s[c + b][1]), kw_hmul2(q4_high(x1), s[c + b][1])};
          add(2 * (c + b) + j, a, hi, lo);
        }
    }
  }

  // The same of 16 fp16 rows.
  __device__ __forceinline__ void values_f16(uint32_t vs, const float (&p)[NT][4]) {
    uint32_t hi[NT][2], lo[NT][2];
    split(p, hi, lo);
    if (!Q4) {
      const int lane = g * 4 + t, r = (lane & 7) + (lane >> 4) * 8, u = lane >> 3 & 1;
#pragma unroll
      for (int m = 0; m < MTILES; m++) {
        uint32_t a[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                     : "r"(vs + f16_off<HD>(r, 2 * m + u)));
        add(m, a, hi, lo);
      }
    } else {
      // elements 2g, 2g + 1 of each half of a block
#pragma unroll
      for (int b = 0; b < BLOCKS; b++) {
        uint32_t v[4][2];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
          for (int h = 0; h < 2; h++)
            v[k][h] = kw_lds32(vs + f16_off<HD>(2 * t + (k & 1) + 8 * (k >> 1), 4 * b + 2 * h + (g >> 2)) + 4 * (g & 3));
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const uint32_t sel = j ? 0x7632 : 0x5410;
          const uint32_t a[4] = {__byte_perm(v[0][0], v[1][0], sel), __byte_perm(v[0][1], v[1][1], sel),
                                 __byte_perm(v[2][0], v[3][0], sel), __byte_perm(v[2][1], v[3][1], sel)};
          add(2 * b + j, a, hi, lo);
        }
      }
    }
  }

  // A tile's values added one key after the other where it holds infinities or NaN
  // that some rows do not see (0 times them is NaN): value(row, dimension).
  template <class F>
  __device__ __forceinline__ void values_slow(const float (&p)[NT][4], F&& value) {
#pragma unroll 1
    for (int k = 0; k < 16; k++) {
      const int src = (k & 7) << 2 | t;
      float pr[NT][2];
      bool any = false;
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const float a = __shfl_sync(0xffffffffu, p[n][h], src), b = __shfl_sync(0xffffffffu, p[n][2 + h], src);
          pr[n][h] = k < 8 ? a : b;
          any |= !(pr[n][h] == 0.0f);
        }
      if (!any) continue;
#pragma unroll
      for (int m = 0; m < MTILES; m++)
#pragma unroll
        for (int half = 0; half < 2; half++) {
          const float v = value(k, dim_of(m, half));
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int h = 0; h < 2; h++)
              if (!(pr[n][h] == 0.0f)) o[m][n][2 * half + h] = fmaf(pr[n][h], v, o[m][n][2 * half + h]);
        }
    }
  }

  // The warp's results: o as x[row][dimension] (rows XROW floats apart), and
  // (maximum, sum) of its rows.
  template <int XROW>
  __device__ __forceinline__ void put(float* x, float2* ml) const {
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float l = sum[n][h];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        const int r = 8 * n + 2 * t + h;
        if (g == 0) ml[r] = make_float2(mx[n][h], l);
#pragma unroll
        for (int m = 0; m < MTILES; m++)
#pragma unroll
          for (int half = 0; half < 2; half++) x[r * XROW + dim_of(m, half)] = o[m][n][2 * half + h];
      }
  }
};

// 32 rows of codes and scales of K and V on their way to a stage (K's codes, V's, K's
// scales, V's) of a warp's ring: lane l has the cache's row `at` of row l, ~0 for zeros.  With
// `runs` the rows of a page come in whole runs of 32: where none is missing they are
// neighbours then.
template <int HD>
__device__ __forceinline__ void load_codes(uint32_t to, uint32_t at, bool runs, const uint8_t* __restrict__ k_qs,
                                           const uint8_t* __restrict__ v_qs, const __half* __restrict__ k_scales,
                                           const __half* __restrict__ v_scales) {
  constexpr int CH = HD / 32, PER = 32 / CH, CODES = 32 * HD / 2, SCALES = 32 * HD / 16;  // chunks of a row, rows a pass
  const int lane = threadIdx.x & 31, c = lane % CH, r = lane / CH;
  const uint32_t ss = to + 2 * CODES + lane * (HD / 16);
  if (runs && __all_sync(0xffffffffu, at != ~0u)) {
    const uint32_t x0 = __shfl_sync(0xffffffffu, at, 0);
    const uint8_t* k = k_qs + (uint64_t)x0 * (HD / 2) + lane * 16;
    const uint8_t* v = v_qs + (uint64_t)x0 * (HD / 2) + lane * 16;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      // (PER is 8 or 16 rows: the swizzle repeats)
      const uint32_t d = to + r * (HD / 2) + ((c ^ q4_swz<HD>(r)) << 4) + i * PER * (HD / 2);
      kw_copy<16>(d, k + i * PER * (HD / 2), true);
      kw_copy<16>(d + CODES, v + i * PER * (HD / 2), true);
    }
    kw_copy<HD / 16>(ss, k_scales + (uint64_t)x0 * CH + lane * CH, true);
    kw_copy<HD / 16>(ss + SCALES, v_scales + (uint64_t)x0 * CH + lane * CH, true);
    return;
  }
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const uint32_t x = __shfl_sync(0xffffffffu, at, i * PER + r);
    const bool ok = x != ~0u;
    const uint64_t from = (uint64_t)(ok ? x : 0u) * (HD / 2) + c * 16;
    const uint32_t d = to + r * (HD / 2) + ((c ^ q4_swz<HD>(r)) << 4) + i * PER * (HD / 2);
    kw_copy<16>(d, k_qs + from, ok);
    kw_copy<16>(d + CODES, v_qs + from, ok);
  }
  const bool ok = at != ~0u;
  const uint64_t from = (uint64_t)(ok ? at : 0u) * CH;
  kw_copy<HD / 16>(ss, k_scales + from, ok);
  kw_copy<HD / 16>(ss + SCALES, v_scales + from, ok);
}

// ---------------------------------------------------------------------------
// the warps' results of a unit, of one CTA or of a cluster's, joined
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_at(uint32_t at, uint32_t rank) {  // the address in another CTA
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}

// The shared memory that a join of WARPS warps a CTA needs: the warps' results over
// whatever has been read (from 0 on), the CTA's behind it.
template <int HD, int ROWS, int WARPS>
struct JoinShape {
  static constexpr int XROW = HD + 4;  // floats of a row (padded)
  static constexpr int PART = ROWS * (XROW * 4 + 8), EXCHANGE = WARPS * PART;
};

// finish(row, unit of 8 dimensions, unnormalised result, sum) for each of `rows` rows of a unit
// which `ranks` (1 to 16, a power of two) CTAs of a cluster have, this one being `rank`: in
// the order of the warps, and of the CTAs by halves.  All threads of all of them; what the
// kernel had in the first EXCHANGE bytes of smem has been read.
template <int WARPS, int HD, int NT, bool Q4, class F>
__device__ __forceinline__ void join_unit(const KeyWarp<HD, NT, Q4>& kw, unsigned char* smem, int part_off, int rank,
                                          int ranks, int rows, F&& finish) {
  constexpr int ROWS = 8 * NT, UNITS = HD / 8, XROW = JoinShape<HD, ROWS, WARPS>::XROW, THREADS = 32 * WARPS;
  const int tid = threadIdx.x, warp = tid >> 5;
  float* x = reinterpret_cast<float*>(smem);
  float2* ml = reinterpret_cast<float2*>(x + (size_t)WARPS * ROWS * XROW);
  float* part = reinterpret_cast<float*>(smem + part_off);
  float2* part_ml = reinterpret_cast<float2*>(part + ROWS * XROW);
  kw.template put<XROW>(x + (size_t)warp * ROWS * XROW, ml + warp * ROWS);
  __syncthreads();
  for (int e = tid; e < rows * UNITS; e += THREADS) {
    const int r = e / UNITS, u = e % UNITS;
    float m2 = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; w++) m2 = fmaxf(m2, ml[w * ROWS + r].x);
    const float ref = m2 == -INFINITY ? 0.0f : m2;
    float acc[8] = {}, l = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; w++) {
      const float2 y = ml[w * ROWS + r];
      const float f = kw_exp2(y.x - ref);
      l = fmaf(y.y, f, l);
      const float4* src = reinterpret_cast<const float4*>(x + ((size_t)w * ROWS + r) * XROW + u * 8);
      const float4 a = src[0], b = src[1];
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int d = 0; d < 8; d++) acc[d] = fmaf(v[d], f, acc[d]);
    }
    if (ranks == 1) {
      finish(r, u, acc, l);
    } else {
      float4* dst = reinterpret_cast<float4*>(part + r * XROW + u * 8);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (u == 0) part_ml[r] = make_float2(m2, l);
    }
  }
  if (ranks == 1) return;
  cluster_sync();
  // a lane a rank: lanes [0, ranks) of a group have one item (row, 8 dimensions)
  const int j = tid & (ranks - 1);
  for (int e0 = 0; e0 < rows * UNITS; e0 += THREADS) {  // items of all ranks together: THREADS a turn
    const int e = e0 + rank * (THREADS / ranks) + tid / ranks;
    const bool ok = e < rows * UNITS;
    const int r = ok ? e / UNITS : 0, u = ok ? e % UNITS : 0;
    const uint32_t from = cluster_at(kw_smem(part + r * XROW + u * 8), j);
    const float2 y = cluster_ld2(cluster_at(kw_smem(part_ml + r), j));
    const float4 v0 = cluster_ld4(from), v1 = cluster_ld4(from + 16);
    float acc[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    float m2 = y.x;
    for (int off = 1; off < ranks; off <<= 1) m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, off));
    const float f = kw_exp2(y.x - (m2 == -INFINITY ? 0.0f : m2));
    float l = y.y * f;
#pragma unroll
    for (int d = 0; d < 8; d++) acc[d] *= f;
    for (int off = 1; off < ranks; off <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
      for (int d = 0; d < 8; d++) acc[d] += __shfl_xor_sync(0xffffffffu, acc[d], off);
    }
    if (ok && j == 0) finish(r, u, acc, l);
  }
  cluster_sync();  // no CTA ends while another one reads its result
}

// Eight dimensions of a finished row.
__device__ __forceinline__ void put_row(__half* to, const float (&acc)[8], float l) {
  const float inv = 1.0f / l;
  *reinterpret_cast<uint4*>(to) =
      make_uint4(kw_pack(acc[0] * inv, acc[1] * inv), kw_pack(acc[2] * inv, acc[3] * inv),
                 kw_pack(acc[4] * inv, acc[5] * inv), kw_pack(acc[6] * inv, acc[7] * inv));
}

// A launch in clusters of `ranks` CTAs, as a programmatic dependent.
template <class A>
inline cudaError_t launch_clusters(void (*kernel)(const A), const A& a, size_t ctas, int threads, int ranks,
                                   size_t smem, cudaStream_t st) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = programmatic_launch() ? 1 : 0;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ranks;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace
