// sample.cu -- one token per row from given random words, after temperature,
// top-k, top-p and min-p (spec_sample).
//
// With the integer weights of the rejection sampler, W_v = floor(exp(z_v -
// max z) * 2^32), every step is integer arithmetic on sums that do not depend
// on their order: the kept set of top-k and top-p is a prefix of the tokens
// ordered by (logit descending, id ascending), so each filter is one cut, the
// (order key, id) of the last token that stays, and the draw is a prefix sum
// of the kept weights in the order of ids.
//
// One cluster of CTAs per row keeps the row in shared memory: the logits are
// read from HBM once, whatever the filters.  A cut is found without sorting
// the row:
//  - top-k: every thread knows the largest of the logits that it loaded; the
//    k-th largest of these is a bound that at least k tokens, and typically
//    few more, reach.  Those are collected and ranked against one another.
//  - top-p alone: a histogram of masses over equal steps of z gives the step
//    that holds the cut; its tokens are collected and ranked.
//  - a step with too many tokens (or a top-k whose bound is reached by too
//    many) is refined by the bits of the order key, down to tokens of equal
//    logits, whose cut is the n-th lowest id.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "sampler.cuh"

namespace cg = cooperative_groups;

namespace {

typedef unsigned long long u64;

constexpr int SM_THREADS = 512;
constexpr int SM_WARPS = SM_THREADS / 32;
constexpr int SM_BINS = 1024;
constexpr int SM_CAND = 2048;   // tokens that are ranked against one another
constexpr int SM_LOCAL = 1024;  // of one CTA
constexpr int SM_MAX_CL = 16;
constexpr float SM_SPAN = 23.0f;  // z steps cover [max - 23, max]: W is 0 from 22.2 below it
// a CTA's logits: the 16-bit halves of as many weights (each below 2^17) sum
// to less than 2^32
constexpr int SM_SEG = 65532;

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
  int V;
  int seg;  // logits of a CTA (a multiple of 4)
  int cap;  // of them in shared memory
};

struct alignas(16) Shared {  // the row's logits (16-byte stores) follow it
  union {
    struct {
      uint32_t cnt[SM_BINS], lo[SM_BINS], hi[SM_BINS];  // counts; masses' low 16 bits, and the rest
    };
    struct {
      u64 own_key[SM_LOCAL];  // this CTA's collected tokens
      uint32_t own_w[SM_LOCAL];
    };
  };
  u64 key[SM_CAND];  // the row's collected tokens: order key, then lower ids first
  uint32_t w[SM_CAND];  // their weights, 2^32 as 2^32 - 1 (which no other weight is)
  u64 slice_w[SM_BINS];       // this rank's share of the combined bins: inclusive sums
  uint32_t slice_c[SM_BINS];
  u64 part[SM_WARPS];
  uint32_t part32[SM_WARPS];
  u64 pub_w;  // this rank's published totals
  uint32_t pub_c;
  uint32_t pub_key;
  int pub_bad;
  uint32_t n_own, theta;
  // published by the rank that finds it
  int f_bin;
  u64 f_before_w;
  uint32_t f_before_c, f_bin_c;
  u64 cut_key, cut_w;
  int pick;
};
static_assert(sizeof(Shared) % 16 == 0, "the logits behind it are 16-byte aligned");

// Inclusive sum of v over the CTA's threads, in thread order; *total: all.
__device__ __forceinline__ u64 block_prefix(u64 v, Shared& sh, u64* total) {
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
  u64 before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < SM_WARPS; w++) {
    const u64 p = sh.part[w];
    if (w < warp) before += p;
    all += p;
  }
  *total = all;
  return before + x;
}

// The row's segment of this CTA.
struct Segment {
  const float* s;  // shared memory: the first `cap` logits
  const float* g;  // global memory
  int len, cap, id0;
  __device__ __forceinline__ float at(int i) const { return i < cap ? s[i] : __ldcg(g + i); }
};

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
  bool plain;  // divide by the division: T is 1 or far from it
  u64 cut;     // tokens whose composite key is at least this stay
  u64 min_w;
  // Order key and id as one number: larger stands first (ties: the lower id).
  static __device__ __forceinline__ u64 composite(float l, int id) {
    return ((u64)max_key(l) << 32) | (uint32_t)~id;
  }
  // x = z - max z of two logits.  z = l / T, correctly rounded: from the
  // correctly rounded reciprocal y of T, q0 = l y; q <- q + (l - q T) y twice.
  // The first step leaves q within one unit in the last place, and the second
  // is then the correctly rounded quotient (Markstein, "Computation of
  // elementary functions on the IBM RISC System/6000 processor", 1990).  Five
  // packed operations for two logits.  Where l / T overflows below, x is NaN,
  // which is taken as a weight of 0 and the last step.
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
  __device__ __forceinline__ bool inside(float l, int id) const { return composite(l, id) >= cut; }
};

// The first id, in the order of ids over the whole row, at which the running
// sum of the two measures of measure(logits, id of the first) reaches
// target(total); every thread of the cluster gets it, and the total.  -1 if
// it is never reached.
template <class M, class Tg>
__device__ int ordered_pick(cg::cluster_group& cl, Shared& sh, const Segment& seg, M&& measure,
                            Tg&& target, u64* total) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  // a thread owns a run of ids; an odd number of pairs keeps its strided
  // reads of shared memory at two wavefronts
  const int c = 2 * (((seg.len + 2 * SM_THREADS - 1) / (2 * SM_THREADS)) | 1);
  const int i0 = min(seg.len, (int)threadIdx.x * c), i1 = min(seg.len, i0 + c);
  auto pair = [&](int i) {  // the second of the last pair may be past the end
    return make_float2(seg.at(i), i + 1 < i1 ? seg.at(i + 1) : -INFINITY);
  };
  u64 mine = 0;
  for (int i = i0; i < i1; i += 2) {
    const ulonglong2 w = measure(pair(i), seg.id0 + i);
    mine += w.x + w.y;
  }
  u64 cta;
  const u64 incl = block_prefix(mine, sh, &cta);
  if (threadIdx.x == 0) {
    sh.pub_w = cta;
    sh.pick = -1;
  }
  cl.sync();
  u64 before = 0, all = 0;
  for (int r = 0; r < n; r++) {
    const u64 w = *cl.map_shared_rank(&sh.pub_w, r);
    if (r < rank) before += w;
    all += w;
  }
  const u64 t = target(all);
  const u64 hi = before + incl, lo = hi - mine;
  if (mine > 0 && lo < t && t <= hi) {  // this thread's run holds it: at most one thread does
    u64 run = lo;
    for (int i = i0; i < i1; i += 2) {
      const ulonglong2 w = measure(pair(i), seg.id0 + i);
      if (run + w.x + w.y >= t) {
        const int id = seg.id0 + i + (run + w.x >= t ? 0 : 1);
        for (int r = 0; r < n; r++) *cl.map_shared_rank(&sh.pick, r) = id;
        break;
      }
      run += w.x + w.y;
    }
  }
  cl.sync();
  *total = all;
  return sh.pick;
}

// The combined bins of the cluster from every CTA's: every rank holds its
// share of them as inclusive sums.
template <bool MASS>
__device__ void combine(cg::cluster_group& cl, Shared& sh) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  cl.sync();
  const int share = SM_BINS / n, b0 = rank * share;
  constexpr int PER = SM_BINS / SM_THREADS;  // bins of a thread at cluster size 1
  u64 w[PER], wt = 0;
  uint32_t ct = 0, cc[PER];
#pragma unroll
  for (int k = 0; k < PER; k++) {
    const int b = (int)threadIdx.x * PER + k;
    w[k] = 0;
    cc[k] = 0;
    if (b < share)
      for (int r = 0; r < n; r++) {
        cc[k] += cl.map_shared_rank(sh.cnt, r)[b0 + b];
        if (MASS)
          w[k] += ((u64)cl.map_shared_rank(sh.hi, r)[b0 + b] << 16) + cl.map_shared_rank(sh.lo, r)[b0 + b];
      }
    wt += w[k];
    ct += cc[k];
  }
  u64 all_w = 0, all_c = 0;
  u64 run_w = MASS ? block_prefix(wt, sh, &all_w) - wt : 0;
  u64 run_c = block_prefix(ct, sh, &all_c) - ct;
#pragma unroll
  for (int k = 0; k < PER; k++) {
    const int b = (int)threadIdx.x * PER + k;
    run_w += w[k];
    run_c += cc[k];
    if (b < share) {
      sh.slice_w[b] = run_w;
      sh.slice_c[b] = (uint32_t)run_c;
    }
  }
  if (threadIdx.x == 0) {
    sh.pub_w = all_w;
    sh.pub_c = (uint32_t)all_c;
  }
  cl.sync();
}

__device__ __forceinline__ void clear_bins(Shared& sh) {
  for (int b = threadIdx.x; b < 3 * SM_BINS; b += SM_THREADS) sh.cnt[b] = 0;  // cnt, lo, hi
  __syncthreads();
}
__device__ __forceinline__ void add_mass(Shared& sh, int b, uint32_t w) {
  const u64 v = widen(w);
  atomicAdd(&sh.lo[b], (uint32_t)v & 0xFFFFu);
  atomicAdd(&sh.hi[b], (uint32_t)(v >> 16));
}

// Histogram of all tokens over the steps of z (two 32-bit additions a mass:
// 64-bit ones in shared memory are compare-and-swap loops, four times slower).
__device__ void histogram(cg::cluster_group& cl, Shared& sh, const Segment& seg, const Row& row) {
  clear_bins(sh);
  for (int i = 2 * threadIdx.x; i < seg.len; i += 2 * SM_THREADS) {
    const bool two = i + 1 < seg.len;
    const float2 x = row.x2(make_float2(seg.at(i), two ? seg.at(i + 1) : -INFINITY));
    const uint2 w = Row::w2(x);
    const int b0 = Row::bin_of(x.x), b1 = Row::bin_of(x.y);
    atomicAdd(&sh.cnt[b0], 1u);
    if (w.x != 0) add_mass(sh, b0, w.x);
    if (two) {
      atomicAdd(&sh.cnt[b1], 1u);
      if (w.y != 0) add_mass(sh, b1, w.y);
    }
  }
  combine<true>(cl, sh);
}

// What a search for a target in the combined bins gives.
struct Found {
  int bin;
  u64 before_w;
  uint32_t before_c, bin_c;
};

// The bin at which the running sum of counts (BY_COUNT) or masses reaches
// `target` (1 <= target <= the total).
template <bool BY_COUNT>
__device__ Found find_bin(cg::cluster_group& cl, Shared& sh, u64 target) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  const int share = SM_BINS / n;
  u64 bw = 0, bc = 0;
  for (int r = 0; r < rank; r++) {
    bw += *cl.map_shared_rank(&sh.pub_w, r);
    bc += *cl.map_shared_rank(&sh.pub_c, r);
  }
  const u64 base = BY_COUNT ? bc : bw;
  for (int b = threadIdx.x; b < share; b += SM_THREADS) {
    const u64 hi = base + (BY_COUNT ? (u64)sh.slice_c[b] : sh.slice_w[b]);
    const u64 lo = base + (b == 0 ? 0ull : BY_COUNT ? (u64)sh.slice_c[b - 1] : sh.slice_w[b - 1]);
    if (lo < target && target <= hi) {
      const u64 pw = b == 0 ? 0ull : sh.slice_w[b - 1];
      const uint32_t pc = b == 0 ? 0u : sh.slice_c[b - 1];
      for (int r = 0; r < n; r++) {
        Shared& o = *cl.map_shared_rank(&sh, r);
        o.f_bin = rank * share + b;
        o.f_before_w = bw + pw;
        o.f_before_c = (uint32_t)bc + pc;
        o.f_bin_c = sh.slice_c[b] - pc;
      }
    }
  }
  cl.sync();
  Found f;
  f.bin = sh.f_bin;
  f.before_w = sh.f_before_w;
  f.before_c = sh.f_before_c;
  f.bin_c = sh.f_bin_c;
  cl.sync();  // read before the next search writes
  return f;
}

struct Cut {
  u64 key;   // composite key of the last token that stays
  u64 mass;  // of the tokens up to it
};

// The tokens that take(logit) accepts, collected into every CTA's sh.key and
// sh.w; returns their number, or more than SM_CAND if they are too many.
template <class P>
__device__ int collect(cg::cluster_group& cl, Shared& sh, const Segment& seg, const Row& row, bool mass,
                       P&& take) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  if (threadIdx.x == 0) sh.n_own = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) {
    const float l = seg.at(i);
    if (take(l)) {
      const uint32_t at = atomicAdd(&sh.n_own, 1u);
      if (at < SM_LOCAL) {
        sh.own_key[at] = Row::composite(l, seg.id0 + i);
        sh.own_w[at] = mass ? row.weight(l) : 0u;
      }
    }
  }
  cl.sync();
  uint32_t before = 0, all = 0;
  bool over = false;
  for (int r = 0; r < n; r++) {
    const uint32_t c = *cl.map_shared_rank(&sh.n_own, r);
    over |= c > SM_LOCAL;
    if (r < rank) before += c;
    all += c;
  }
  if (!over && all <= SM_CAND) {
    const int own = (int)sh.n_own;
    for (int e = threadIdx.x; e < own * n; e += SM_THREADS) {
      const int r = e / own, c = e - r * own;
      Shared& o = *cl.map_shared_rank(&sh, r);
      o.key[before + c] = sh.own_key[c];
      o.w[before + c] = sh.own_w[c];
    }
  }
  cl.sync();
  return over ? SM_CAND + 1 : (int)all;
}

// Ranks the m collected tokens against one another, each by up to 32 threads
// of the CTAs in turn, and calls f(composite key, count and mass in front of
// it, weight) once for each, on some thread of the cluster.
template <class F>
__device__ void rank_all(cg::cluster_group& cl, Shared& sh, int m, bool mass, F&& f) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  const int per = (m + n - 1) / n, c0 = rank * per, mine = max(0, min(m - c0, per));
  int grp = 1;  // threads of a token
  while (grp < 32 && mine * grp * 2 <= SM_THREADS) grp *= 2;
  const int step = SM_THREADS / grp;
  for (int base = 0; base < mine; base += step) {  // uniform over the CTA
    const int c = base + (int)threadIdx.x / grp;
    const bool ok = c < mine;
    const u64 me = ok ? sh.key[c0 + c] : ~0ull;
    uint32_t cnt = 0;
    u64 sum = 0;
    if (mass) {
      for (int j = threadIdx.x % grp; j < m; j += grp)
        if (sh.key[j] > me) {
          cnt++;
          sum += widen(sh.w[j]);
        }
    } else {
      for (int j = threadIdx.x % grp; j < m; j += grp) cnt += sh.key[j] > me;
    }
    for (int off = grp >> 1; off > 0; off >>= 1) {
      cnt += __shfl_xor_sync(0xffffffffu, cnt, off);
      sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
    if (ok && threadIdx.x % grp == 0) f(me, cnt, sum, widen(sh.w[c0 + c]));
  }
}

__device__ __forceinline__ void publish(cg::cluster_group& cl, Shared& sh, u64 key, u64 mass) {
  for (int r = 0; r < (int)cl.num_blocks(); r++) {
    Shared& o = *cl.map_shared_rank(&sh, r);
    o.cut_key = key;
    o.cut_w = mass;
  }
}

// The token at which the running sum of counts (BY_COUNT) or masses, in the
// order (logit descending, id ascending), reaches `target`.  The histogram of
// all tokens over the steps of z is combined; the search overwrites it.
template <bool BY_COUNT>
__device__ Cut find_cut(cg::cluster_group& cl, Shared& sh, const Segment& seg, const Row& row,
                        u64 target) {
  Found f = find_bin<BY_COUNT>(cl, sh, target);
  const int zbin = f.bin;
  u64 before_w = f.before_w;
  u64 left = target - (BY_COUNT ? (u64)f.before_c : f.before_w);  // to reach inside the bin
  uint32_t members = f.bin_c;
  // refinement by the bits of the order key: 10, 10, 10, 2 from the top,
  // larger keys in lower bins
  int known = 32;  // bits still unknown
  uint32_t prefix = 0;
  auto member = [&](float l, uint32_t k) {
    return (known >= 32 || (k >> known) == prefix) && row.bin(l) == zbin;
  };
  int m = SM_CAND + 1;
  for (;;) {
    if (members <= SM_CAND) m = collect(cl, sh, seg, row, true, [&](float l) { return member(l, max_key(l)); });
    if (m <= SM_CAND || known == 0) break;
    const int bits = min(10, known), down = known - bits;
    clear_bins(sh);
    for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) {
      const float l = seg.at(i);
      const uint32_t k = max_key(l);
      if (member(l, k)) {
        const int b = (SM_BINS - 1) - (int)((k >> down) & ((1u << bits) - 1u));
        atomicAdd(&sh.cnt[b], 1u);
        add_mass(sh, b, row.weight(l));
      }
    }
    combine<true>(cl, sh);
    f = find_bin<BY_COUNT>(cl, sh, left);
    before_w += f.before_w;
    left -= BY_COUNT ? (u64)f.before_c : f.before_w;
    prefix = (known < 32 ? prefix << bits : 0u) | (uint32_t)((SM_BINS - 1) - f.bin);
    known = down;
    members = f.bin_c;
  }
  Cut cut;
  if (m > SM_CAND) {  // all of one logit: the n-th lowest id of them
    const uint32_t key = prefix;
    const u64 w = widen(row.weight(key_value(key)));
    const u64 nth = BY_COUNT ? left : (left + w - 1) / w;
    u64 all;
    const int id = ordered_pick(
        cl, sh, seg,
        [&](float2 l, int) { return make_ulonglong2(max_key(l.x) == key, max_key(l.y) == key); },
        [&](u64) { return nth; }, &all);
    cut.key = ((u64)key << 32) | (uint32_t)~id;
    cut.mass = before_w + nth * w;
    return cut;
  }
  rank_all(cl, sh, m, true, [&](u64 key, uint32_t cnt, u64 sum, u64 w) {
    const u64 lo = BY_COUNT ? (u64)cnt : sum, step = BY_COUNT ? 1ull : w;
    if (lo < left && left <= lo + step) publish(cl, sh, key, before_w + sum + w);
  });
  cl.sync();
  cut.key = sh.cut_key;
  cut.mass = sh.cut_w;
  cl.sync();  // read before the next search writes
  return cut;
}

// The first token at which the mass reaches P / 2^32 of S.
__device__ __forceinline__ u64 mass_needed(u64 P, u64 S) {
  const u64 need = (u64)(((u128)P * S + 0xFFFFFFFFull) >> 32);
  return need == 0 ? 1 : need;
}

__global__ void __launch_bounds__(SM_THREADS, 2)
sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  Shared& sh = *reinterpret_cast<Shared*>(dyn);
  float* buf = reinterpret_cast<float*>(dyn + sizeof(Shared));
  cg::cluster_group cl = cg::this_cluster();
  const int n = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int r = blockIdx.x / n;
  const float* grow = a.logits + (int64_t)r * a.ld;
  Segment seg;
  seg.id0 = min(a.V, rank * a.seg);
  seg.len = min(a.V, seg.id0 + a.seg) - seg.id0;
  seg.g = grow + seg.id0;
  seg.s = buf;
  seg.cap = min(a.cap, seg.len);
  Row row;
  row.T = a.temperature != nullptr ? a.temperature[r] : 1.0f;
  int k = a.top_k != nullptr ? a.top_k[r] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[r] : 1.0f;
  const float min_p = a.min_p != nullptr ? a.min_p[r] : 0.0f;
  bool bad = !(row.T >= 0.0f && row.T <= FLT_MAX) || k < 0 || !(top_p >= 0.0f && top_p <= 1.0f) ||
             !(min_p >= 0.0f && min_p <= 1.0f);
  if (row.T == 0.0f) {  // greedy: the first of the order
    row.T = 1.0f;
    k = 1;
  }
  if (bad) row.T = 1.0f;
  row.inv_T = __frcp_rn(row.T);
  row.plain = row.T == 1.0f || !(row.T > 0x1p-60f && row.T < 0x1p60f);

  // ---- the segment into shared memory; its largest logit, NaN and +inf
  float mx = -INFINITY;  // of this thread's
  bool nan = false;
  int finite = 0;  // logits above -inf
  auto see = [&](float l) {
    nan |= !(l < INFINITY);
    finite += l > -INFINITY;
    mx = fmaxf(mx, l);
  };
  if ((reinterpret_cast<uintptr_t>(seg.g) & 15u) == 0) {
    const int n4 = seg.cap / 4;
    const float4* g4 = reinterpret_cast<const float4*>(seg.g);
    constexpr int U = 8;
    for (int i = threadIdx.x; i < n4; i += SM_THREADS * U) {
      float4 t[U];
#pragma unroll
      for (int v = 0; v < U; v++)
        if (i + v * SM_THREADS < n4) t[v] = __ldcs(g4 + i + v * SM_THREADS);
#pragma unroll
      for (int v = 0; v < U; v++)
        if (i + v * SM_THREADS < n4) {
          reinterpret_cast<float4*>(buf)[i + v * SM_THREADS] = t[v];
          see(t[v].x), see(t[v].y), see(t[v].z), see(t[v].w);
        }
    }
    for (int i = 4 * n4 + threadIdx.x; i < seg.cap; i += SM_THREADS) see(buf[i] = seg.g[i]);
  } else {
#pragma unroll 8
    for (int i = threadIdx.x; i < seg.cap; i += SM_THREADS) see(buf[i] = seg.g[i]);
  }
  for (int i = seg.cap + threadIdx.x; i < seg.len; i += SM_THREADS) see(__ldcg(seg.g + i));
  float cmx = mx;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    cmx = fmaxf(cmx, __shfl_xor_sync(0xffffffffu, cmx, off));
    finite += __shfl_xor_sync(0xffffffffu, finite, off);
  }
  if ((threadIdx.x & 31) == 0) {
    sh.part32[threadIdx.x >> 5] = max_key(cmx);
    sh.part[threadIdx.x >> 5] = finite;
  }
  const int any_nan = __syncthreads_or(nan);
  if (threadIdx.x == 0) {
    uint32_t key = 0, fin = 0;
    for (int w = 0; w < SM_WARPS; w++) {
      key = max(key, sh.part32[w]);
      fin += (uint32_t)sh.part[w];
    }
    sh.pub_key = key;
    sh.pub_bad = any_nan;
    sh.pub_c = fin;
  }
  cl.sync();
  uint32_t key = 0, n_fin = 0;
  for (int q = 0; q < n; q++) {
    key = max(key, *cl.map_shared_rank(&sh.pub_key, q));
    bad |= *cl.map_shared_rank(&sh.pub_bad, q) != 0;
    n_fin += *cl.map_shared_rank(&sh.pub_c, q);
  }
  cl.sync();  // read before the next totals are published
  row.zmax = row_zmax(key, row.T);
  bad |= n_fin == 0 || !(fabsf(row.zmax) < INFINITY);
  float* frow = a.filtered != nullptr ? a.filtered + (int64_t)r * a.ldf + seg.id0 : nullptr;
  if (bad) {  // the whole cluster
    if (frow != nullptr)
      for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) frow[i] = __int_as_float(0x7FFFFFFF);
    if (rank == 0 && threadIdx.x == 0) {
      a.token[r] = -1;
      if (a.n_kept != nullptr) a.n_kept[r] = 0;
    }
    return;
  }

  // ---- the cuts.  Everything above -inf is inside at first.
  row.cut = (u64)0x00800000u << 32;  // the key of -FLT_MAX, any id
  row.min_w = (u64)floor((double)min_p * 4294967296.0);
  const u64 P = (u64)floor((double)top_p * 4294967296.0);
  const bool by_k = k > 0 && (uint32_t)k < n_fin, by_p = P < (1ull << 32);
  bool done = false;
  if (by_k && k <= n * SM_THREADS) {
    // the k-th largest of the threads' largest logits, to a step of z: no
    // token below it is among the first k
    clear_bins(sh);
    if (mx > -INFINITY) atomicAdd(&sh.cnt[row.bin(mx)], 1u);
    if (threadIdx.x == 0) sh.theta = ~0u;
    combine<false>(cl, sh);
    uint32_t threads = 0;  // with a finite logit
    for (int q = 0; q < n; q++) threads += *cl.map_shared_rank(&sh.pub_c, q);
    if ((uint32_t)k <= threads) {
      const Found f = find_bin<true>(cl, sh, (u64)k);
      if (mx > -INFINITY && row.bin(mx) <= f.bin) atomicMin(&sh.theta, max_key(mx));
      cl.sync();
      uint32_t theta = ~0u;
      for (int q = 0; q < n; q++) theta = min(theta, *cl.map_shared_rank(&sh.theta, q));
      const float bound = key_value(theta);
      const int m = collect(cl, sh, seg, row, by_p, [&](float l) { return l >= bound; });
      if (m <= SM_CAND) {
        // a thread ranks at most SM_CAND / SM_THREADS tokens; the cut of the
        // mass needs the total up to the k-th first
        u64 keys[SM_CAND / SM_THREADS], sums[SM_CAND / SM_THREADS], ws[SM_CAND / SM_THREADS];
        int held = 0;
#pragma unroll
        for (int e = 0; e < SM_CAND / SM_THREADS; e++) keys[e] = sums[e] = ws[e] = 0;
        rank_all(cl, sh, m, by_p, [&](u64 ck, uint32_t cnt, u64 sum, u64 w) {
#pragma unroll
          for (int e = 0; e < SM_CAND / SM_THREADS; e++)
            if (e == held) keys[e] = ck, sums[e] = sum, ws[e] = w;
          held++;
          if (cnt == (uint32_t)k - 1) publish(cl, sh, ck, sum + w);
        });
        cl.sync();
        row.cut = sh.cut_key;
        const u64 S = sh.cut_w;
        cl.sync();
        if (by_p) {
          const u64 need = mass_needed(P, S);
#pragma unroll
          for (int e = 0; e < SM_CAND / SM_THREADS; e++)
            if (e < held && sums[e] < need && need <= sums[e] + ws[e]) publish(cl, sh, keys[e], 0);
          cl.sync();
          row.cut = sh.cut_key;
        }
        done = true;
      }
    }
  }
  if (!done && (by_k || by_p)) {
    u64 S = 0;
    histogram(cl, sh, seg, row);
    if (by_p && !by_k)
      for (int q = 0; q < n; q++) S += *cl.map_shared_rank(&sh.pub_w, q);
    if (by_k) {
      const Cut c = find_cut<true>(cl, sh, seg, row, (u64)k);
      row.cut = c.key;
      S = c.mass;
      if (by_p) histogram(cl, sh, seg, row);
    }
    if (by_p) row.cut = find_cut<false>(cl, sh, seg, row, mass_needed(P, S)).key;
  }

  // ---- the draw, in the order of ids
  const uint32_t u = a.u[r];
  u64 total;
  const float least = key_value((uint32_t)(row.cut >> 32));  // logits below it are outside
  const int tok = ordered_pick(
      cl, sh, seg,
      [&](float2 l, int id) {
        ulonglong2 w = make_ulonglong2(0, 0);
        if (l.x >= least || l.y >= least) {
          const uint2 v = row.weight2(l);
          if (row.inside(l.x, id) && widen(v.x) >= row.min_w) w.x = widen(v.x);
          if (row.inside(l.y, id + 1) && widen(v.y) >= row.min_w) w.y = widen(v.y);
        }
        return w;
      },
      [&](u64 all) { return (u64)scaled_threshold(u, all) + 1; }, &total);
  if (rank == 0 && threadIdx.x == 0) a.token[r] = tok;
  if (a.n_kept == nullptr && frow == nullptr) return;
  int kept = 0;
  auto stays = [&](float l, int id) {
    return l >= least && row.inside(l, id) && (row.min_w == 0 || widen(row.weight(l)) >= row.min_w);
  };
  if (frow != nullptr && (reinterpret_cast<uintptr_t>(frow) & 15u) == 0 && seg.cap == seg.len) {
    const int n4 = seg.len / 4;
    for (int i = threadIdx.x; i < n4; i += SM_THREADS) {
      float4 l = reinterpret_cast<const float4*>(buf)[i];
      const int id = seg.id0 + 4 * i;
      const bool s0 = stays(l.x, id), s1 = stays(l.y, id + 1), s2 = stays(l.z, id + 2), s3 = stays(l.w, id + 3);
      kept += s0 + s1 + s2 + s3;
      l = make_float4(s0 ? l.x : SPEC_FILTERED, s1 ? l.y : SPEC_FILTERED, s2 ? l.z : SPEC_FILTERED,
                      s3 ? l.w : SPEC_FILTERED);
      __stcs(reinterpret_cast<float4*>(frow) + i, l);
    }
    for (int i = 4 * n4 + threadIdx.x; i < seg.len; i += SM_THREADS) {
      const bool s0 = stays(buf[i], seg.id0 + i);
      kept += s0;
      frow[i] = s0 ? buf[i] : SPEC_FILTERED;
    }
  } else {
    for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) {
      const float l = seg.at(i);
      const bool s0 = stays(l, seg.id0 + i);
      kept += s0;
      if (frow != nullptr) frow[i] = s0 ? l : SPEC_FILTERED;
    }
  }
  if (a.n_kept != nullptr) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) kept += __shfl_xor_sync(0xffffffffu, kept, off);
    if ((threadIdx.x & 31) == 0) sh.part32[threadIdx.x >> 5] = (uint32_t)kept;
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t all = 0;
      for (int w = 0; w < SM_WARPS; w++) all += sh.part32[w];
      sh.pub_c = all;
    }
    cl.sync();
    if (rank == 0 && threadIdx.x == 0) {
      uint32_t all = 0;
      for (int q = 0; q < n; q++) all += *cl.map_shared_rank(&sh.pub_c, q);
      a.n_kept[r] = (int)all;
    }
    cl.sync();  // shared memory stays until rank 0 has read it
  }
}

}  // namespace
void sample_init_attrs() {
  int dev = 0, optin = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
  cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

int launch_sample(const float* logits, int R, int V, int64_t ld, const uint32_t* u,
                  const float* temperature, const int32_t* top_k, const float* top_p,
                  const float* min_p, int32_t* token, int32_t* n_kept, float* filtered, int64_t ldf,
                  cudaStream_t st) {
  SampleArgs a;
  a.logits = logits;
  a.ld = ld;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.token = token;
  a.n_kept = n_kept;
  a.filtered = filtered;
  a.ldf = ldf;
  a.V = V;
  // CTAs of a row: with 8192 logits each (16384 where the rows alone fill the
  // SMs) a row's CTAs leave room for another cluster's beside them, whose
  // loads go on while these compute
  int cl = 1;
  const int each = (long long)R * SM_MAX_CL > 1024 ? 16384 : 4096;
  while (cl < SM_MAX_CL && V > each * cl) cl *= 2;
  a.seg = ((V + cl - 1) / cl + 3) / 4 * 4;
  if (a.seg > SM_SEG) return fail(SPEC_E_SHAPE, "V above 1048512 is not supported");
  const int room = (int)((227 * 1024 - sizeof(Shared)) / sizeof(float)) / 4 * 4;
  a.cap = std::min(a.seg, room);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cl;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)R * cl);
  cfg.blockDim = dim3(SM_THREADS);
  cfg.dynamicSmemBytes = sizeof(Shared) + sizeof(float) * (size_t)a.cap;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sample_kernel, a);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("sample: ") + cudaGetErrorString(e));
  return SPEC_OK;
}
