// sample.cuh -- what the two forms of the filtered sampling share (sample.cu: a
// cluster per row; sample_rows.cu: passes over many rows): arguments, a row's
// weights, the selection among collected tokens.  Internal.
#pragma once

#include <float.h>
#include <math.h>

#include "common.cuh"
#include "sampler.cuh"

typedef unsigned long long u64;

struct SampleArgs {
  const float* logits;
  int64_t ld;
  const uint32_t* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* token;
  int32_t* n_kept;
  float* filtered;
  int64_t ldf;
  int R, V;
  // rows of `rows` (its first *n_rows) instead of 0 .. R - 1, if not NULL
  const int32_t* rows;
  const int32_t* n_rows;
  int seg;  // logits of a CTA (a multiple of 4)
  int cap;  // of them in shared memory
};

// Launches: the cluster per row, and the passes with their workspace.
int sample_clusters_launch(SampleArgs a, int clusters, cudaStream_t st);
size_t sample_rows_bytes(int R, int V);
int sample_rows_launch(SampleArgs a, void* workspace, cudaStream_t st);
void sample_rows_init_attrs();

namespace {

constexpr int SM_THREADS = 512;
constexpr int SM_WARPS = SM_THREADS / 32;
constexpr int SM_BINS = 1024;
constexpr int SM_CAND = 2048;   // tokens that are collected
constexpr int SM_LOCAL = 1024;  // of one CTA
constexpr int SM_MAX_CL = 16;
constexpr int SM_GROUPS = SM_THREADS / 4;  // of a CTA: four threads each
constexpr float SM_SPAN = 23.0f;  // z steps cover [max - 23, max]: W is 0 from 22.2 below it
// a CTA's logits: the 16-bit halves of as many weights (each below 2^17) sum
// to less than 2^32
constexpr int SM_SEG = 65532;

struct Cut {
  u64 key;   // composite key of the last token that stays
  u64 mass;  // of the tokens up to it
};

// What a CTA keeps in shared memory to find a cut among collected tokens.
struct ListSmem {
  union {
    struct {
      uint32_t cnt[SM_BINS], lo[SM_BINS], hi[SM_BINS];  // counts; masses' low 16 bits, and the rest
    };
    u64 own_key[SM_LOCAL];  // this CTA's collected tokens
  };
  u64 part[SM_WARPS];
  uint32_t part32[4 * SM_WARPS];
  Cut cut;
  u64 list_lo, list_w;
  uint32_t list_c;
  int list_bin;
};

// Inclusive sum of v over the CTA's threads, in thread order; *total: all.
__device__ __forceinline__ u64 block_prefix(u64 v, ListSmem& sh, u64* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 31) sh.part[warp] = x;
  __syncthreads();
  // every warp adds the warps' sums up, a lane one of them
  u64 p = lane < SM_WARPS ? sh.part[lane] : 0;
  const u64 own = p;
#pragma unroll
  for (int off = 1; off < SM_WARPS; off <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, p, off);
    if (lane >= off) p += y;
  }
  *total = __shfl_sync(0xffffffffu, p, SM_WARPS - 1);
  return __shfl_sync(0xffffffffu, p - own, warp) + x;
}

// --- two floats at a time; each product and sum is rounded as a scalar one ----
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ u64 widen(uint32_t w) { return (u64)w + (w == 0xFFFFFFFFu); }

// One row's state in registers of every thread.
struct Row {
  float T, inv_T, zmax;
  bool plain;  // divide by the division: T is 1 or far from it, or a quotient may be at the end of the range
  float least;  // tokens above it stay; those equal to it with ids up to last_id
  int last_id;
  uint32_t min_w;  // of those, the ones of at least this weight (2^32 as 2^32 - 1)
  // Order key and id (20 bits) as one number, larger for what stands first
  // (of equal logits the lower id).
  static __device__ __forceinline__ u64 composite(uint32_t key, int id) {
    return ((u64)key << 20) | (uint32_t)(0xFFFFF - id);
  }
  // x = z - max z of two logits.  z = l / T, correctly rounded: from the
  // correctly rounded reciprocal y of T, q0 = l y; q <- q + (l - q T) y twice.
  // The first step leaves q within one unit in the last place, and the second
  // is then the correctly rounded quotient (Markstein, "Computation of
  // elementary functions on the IBM RISC System/6000 processor", 1990).  Five
  // packed operations for two logits.  Where l / T overflows below, x is NaN,
  // which is taken as a weight of 0 and the last step.  l y may overflow where
  // l / T is within two units of the largest float, so rows whose largest z is
  // far are divided by the division; in the others such a z lies so far below
  // the largest that its weight is 0 and its step the last all the same.
  static __device__ __forceinline__ bool far(float z) { return fabsf(z) > 0x1p126f; }
  __device__ __forceinline__ float2 x2(float2 l) const {
    float2 z;
    if (plain) {
      z = make_float2(zval(l.x, T), zval(l.y, T));
    } else {
      const float2 y = both(inv_T), nT = both(-T);
      z = mul2(l, y);
      z = fma2(fma2(z, nT, l), y, z);
      z = fma2(fma2(z, nT, l), y, z);
    }
    return add2(z, both(-zmax));
  }
  // int_weight of two x, as 32 bits (2^32 as 2^32 - 1).  The same roundings:
  // n times the 15-bit part of ln 2 is exact, so that its subtraction may be
  // fused; the rounding to a whole number is an addition of 1.5 2^23; below
  // -87 the weight is 0 at -87 already.
  static __device__ __forceinline__ uint2 w2(float2 x) {
    const float LOG2E = 0x1.715476p+0f, LN2_HI = 0x1.62e4p-1f, LN2_LO = 0x1.7f7d1cp-20f;
    const float C[8] = {0x1p+0f,        0x1p+0f,        0x1p-1f,         0x1.555556p-3f,
                        0x1.555556p-5f, 0x1.111112p-7f, 0x1.6c16c2p-10f, 0x1.a01a02p-13f};
    const float MAGIC = 0x1.8p+23f;
    x.x = fmaxf(x.x, -87.0f);
    x.y = fmaxf(x.y, -87.0f);
    const float2 t = add2(mul2(x, both(LOG2E)), both(MAGIC)), n = add2(t, both(-MAGIC));
    float2 r = fma2(n, both(-LN2_HI), x);
    const float2 low = mul2(n, both(-LN2_LO));
    r = add2(r, low);
    float2 p = both(C[7]);
#pragma unroll
    for (int k = 6; k >= 0; k--) p = add2(mul2(p, r), both(C[k]));
    // 2^(n + 32) from the low bits of t
    const int ex = __float_as_int(t.x), ey = __float_as_int(t.y);
    constexpr int BASE = 0x4B400000;  // bits of MAGIC
    const float2 v = mul2(p, make_float2(__int_as_float((ex - BASE + 159) << 23), __int_as_float((ey - BASE + 159) << 23)));
    return make_uint2(__float2uint_rz(v.x), __float2uint_rz(v.y));  // saturates 2^32
  }
  __device__ __forceinline__ uint2 weight2(float2 l) const { return w2(x2(l)); }
  __device__ __forceinline__ uint32_t weight(float l) const { return weight2(make_float2(l, l)).x; }
  static __device__ __forceinline__ int bin_of(float x) {
    const float b = x * (-(float)SM_BINS / SM_SPAN);  // +inf for a logit of -inf
    return b < (float)(SM_BINS - 1) ? (int)b : SM_BINS - 1;
  }
  __device__ __forceinline__ int bin(float l) const { return bin_of(x2(make_float2(l, l)).x); }
  __device__ __forceinline__ void set_cut(u64 key) {
    least = key_value((uint32_t)(key >> 20));
    last_id = 0xFFFFF - (int)(key & 0xFFFFFu);
    if (!(least > -INFINITY)) no_cut();  // a top-k beyond the finite logits
  }
  __device__ __forceinline__ void no_cut() {
    least = -FLT_MAX;
    last_id = 0x7FFFFFFF;
  }
  __device__ __forceinline__ bool inside(float l, int id) const {
    return l > least || (l == least && id <= last_id);
  }
};

__device__ __forceinline__ void add_mass(ListSmem& sh, int b, uint32_t w) {
  const u64 v = widen(w);
  atomicAdd(&sh.lo[b], (uint32_t)v & 0xFFFFu);
  atomicAdd(&sh.hi[b], (uint32_t)(v >> 16));
}

// Of the m collected tokens (their keys and weights in shared memory), the one at which the running count or mass, in
// the order of their composite keys, reaches `target`; `mass` gets the sum of
// the masses up to it.  Radix selection, nine bits a step, from the first of
// the `open` low bits in which the keys may differ (prefix: those above);
// ends at the first step that leaves one token.
constexpr int LIST_BITS = 9, LIST_BINS = 1 << LIST_BITS;
static_assert(LIST_BINS == SM_THREADS, "a bin a thread");
__device__ Cut cut_list(ListSmem& sh, const u64* keys, const uint32_t* ws, int m, bool by_count, bool masses,
                        u64 target, int open, u64 prefix) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  u64 left = target, before = 0;
  while (open > 0) {
    const int down = max(0, open - LIST_BITS), bits = open - down;
    sh.cnt[tid] = 0u;
    if (masses) sh.lo[tid] = sh.hi[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < m; i += SM_THREADS) {
      const u64 key = keys[i];
      if ((key >> open) == prefix) {
        const int b = LIST_BINS - 1 - (int)((key >> down) & ((1u << bits) - 1u));
        atomicAdd(&sh.cnt[b], 1u);
        if (masses) add_mass(sh, b, ws[i]);
      }
    }
    __syncthreads();
    const uint32_t c = sh.cnt[tid];
    const u64 w = masses ? ((u64)sh.hi[tid] << 16) + sh.lo[tid] : 0;
    uint32_t rc = c;
    u64 rw = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, rc, off);
      if (lane >= off) rc += x;
    }
    if (masses)
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, rw, off);
        if (lane >= off) rw += y;
      }
    if (lane == 31) {
      sh.part32[warp] = rc;
      sh.part[warp] = rw;
    }
    __syncthreads();
    rc += __reduce_add_sync(0xffffffffu, lane < warp ? sh.part32[lane] : 0u);
    if (masses) {
      u64 front = lane < warp ? sh.part[lane] : 0;
#pragma unroll
      for (int off = SM_WARPS / 2; off > 0; off >>= 1) front += __shfl_xor_sync(0xffffffffu, front, off);
      rw += __shfl_sync(0xffffffffu, front, 0);
    }
    const u64 hi = by_count ? rc : rw, lo = hi - (by_count ? c : w);
    if (lo < left && left <= hi) {
      sh.list_bin = tid;
      sh.list_lo = lo;
      sh.list_w = rw - w;
      sh.list_c = c;
    }
    __syncthreads();
    prefix = (prefix << bits) | (u64)(LIST_BINS - 1 - sh.list_bin);
    left -= sh.list_lo;
    before += sh.list_w;
    open = down;
    if (sh.list_c == 1) break;
  }
  for (int i = tid; i < m; i += SM_THREADS)
    if ((keys[i] >> open) == prefix) {  // one token
      sh.cut.key = keys[i];
      sh.cut.mass = before + (masses ? widen(ws[i]) : 0);
    }
  __syncthreads();
  const Cut c = sh.cut;
  __syncthreads();
  return c;
}

// The first token at which the mass reaches P / 2^32 of S.
__device__ __forceinline__ u64 mass_needed(u64 P, u64 S) {
  const u64 need = (u64)(((u128)P * S + 0xFFFFFFFFull) >> 32);
  return need == 0 ? 1 : need;
}

}  // namespace
