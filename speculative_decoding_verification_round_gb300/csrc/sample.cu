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
// read from HBM once, whatever the filters.  The cut of a target (a count for
// top-k, a mass for top-p) is found without sorting: a histogram of counts
// and masses over equal steps of z, combined over the cluster, gives the bin
// that holds the target; its tokens (typically a few hundred) are collected
// and the one that reaches the target is found by ranking them against one
// another.  A bin with too many tokens is refined by its order keys' bits
// first, down to tokens of equal logits, whose cut is the n-th lowest id.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "sampler.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int SM_THREADS = 512;
constexpr int SM_WARPS = SM_THREADS / 32;
constexpr int SM_BINS = 2048;
constexpr int SM_CAND = 1024;  // tokens that are ranked against one another
constexpr int SM_MAX_CL = 8;
constexpr float SM_SPAN = 23.0f;  // z steps cover [max - 23, max]: W is 0 from 22.2 below it

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

typedef unsigned long long u64;

struct Cand {
  uint32_t key;
  int id;
  u64 w;
};

struct alignas(16) Shared {  // the row's logits (16-byte stores) follow it
  u64 wsum[SM_BINS];
  uint32_t cnt[SM_BINS];
  u64 slice_w[SM_BINS];      // this rank's share of the combined bins: inclusive sums
  uint32_t slice_c[SM_BINS];
  Cand cand[SM_CAND];        // of rank 0
  u64 part[SM_WARPS];
  uint32_t part32[SM_WARPS];
  u64 pub_w;       // this rank's published totals
  uint32_t pub_c;
  uint32_t pub_key;
  int pub_bad;
  // published by the rank that finds it
  int f_bin;
  u64 f_before_w, f_bin_w;
  uint32_t f_before_c, f_bin_c;
  uint32_t n_cand;  // of rank 0
  uint32_t cut_key;
  int cut_id;
  u64 cut_w;  // mass up to and with the cut
  int pick;
  int owner;
  u64 owner_before;
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

// One row's state in registers of every thread.
struct Row {
  float T, zmax;
  uint32_t cut_key;  // tokens with a larger key, or this key and an id up to cut_id, stay
  int cut_id;
  u64 min_w;
  __device__ __forceinline__ float x(float l) const { return __fsub_rn(zval(l, T), zmax); }
  __device__ __forceinline__ u64 weight(float l) const { return int_weight(x(l)); }
  __device__ __forceinline__ int bin(float l) const {
    const float b = __fmul_rn(-x(l), (float)SM_BINS / SM_SPAN);  // +inf for a logit of -inf
    return b < (float)(SM_BINS - 1) ? (int)b : SM_BINS - 1;
  }
  __device__ __forceinline__ bool inside(float l, int id) const {
    const uint32_t k = max_key(l);
    return k > cut_key || (k == cut_key && id <= cut_id);
  }
};

// The first id, in the order of ids over the whole row, at which the running
// sum of measure(l, id) reaches target(total); every thread of the cluster
// gets it, and the total.  -1 if it is never reached.
template <class M, class Tg>
__device__ int ordered_pick(cg::cluster_group& cl, Shared& sh, const Segment& seg, M&& measure,
                            Tg&& target, u64* total) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  // a thread owns a run of ids; its odd length keeps the strided reads of
  // shared memory free of bank conflicts
  const int c = ((seg.len + SM_THREADS - 1) / SM_THREADS) | 1;
  const int i0 = min(seg.len, (int)threadIdx.x * c), i1 = min(seg.len, i0 + c);
  u64 mine = 0;
  for (int i = i0; i < i1; i++) mine += measure(seg.at(i), seg.id0 + i);
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
    for (int i = i0; i < i1; i++) {
      run += measure(seg.at(i), seg.id0 + i);
      if (run >= t) {
        for (int r = 0; r < n; r++) *cl.map_shared_rank(&sh.pick, r) = seg.id0 + i;
        break;
      }
    }
  }
  cl.sync();
  *total = all;
  return sh.pick;
}

// Histogram of the tokens that `take` gives a bin (>= 0), combined over the
// cluster: every rank holds its share of the bins as inclusive sums.
template <bool COUNT, bool MASS, class B>
__device__ void histogram(cg::cluster_group& cl, Shared& sh, const Segment& seg, const Row& row,
                          B&& take) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  for (int b = threadIdx.x; b < SM_BINS; b += SM_THREADS) {
    sh.cnt[b] = 0;
    sh.wsum[b] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) {
    const float l = seg.at(i);
    const int b = take(l);
    if (b >= 0) {
      if (COUNT) atomicAdd(&sh.cnt[b], 1u);
      if (MASS) {
        const u64 w = row.weight(l);
        if (w != 0) atomicAdd(&sh.wsum[b], w);
      }
    }
  }
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
        if (COUNT) cc[k] += cl.map_shared_rank(sh.cnt, r)[b0 + b];
        if (MASS) w[k] += cl.map_shared_rank(sh.wsum, r)[b0 + b];
      }
    wt += w[k];
    ct += cc[k];
  }
  u64 all_w = 0, all_c = 0;
  u64 run_w = MASS ? block_prefix(wt, sh, &all_w) - wt : 0;
  u64 run_c = COUNT ? block_prefix(ct, sh, &all_c) - ct : 0;
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

// What a search for a target in the combined bins gives.
struct Found {
  int bin;
  u64 before_w, bin_w;
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
        o.f_bin_w = sh.slice_w[b] - pw;
        o.f_before_c = (uint32_t)bc + pc;
        o.f_bin_c = sh.slice_c[b] - pc;
      }
    }
  }
  cl.sync();
  Found f;
  f.bin = sh.f_bin;
  f.before_w = sh.f_before_w;
  f.bin_w = sh.f_bin_w;
  f.before_c = sh.f_before_c;
  f.bin_c = sh.f_bin_c;
  cl.sync();  // read before the next search writes
  return f;
}

struct Cut {
  uint32_t key;
  int id;
  u64 mass;  // of the tokens up to it
};

// The token at which the running sum of counts (BY_COUNT) or masses, in the
// order (logit descending, id ascending), reaches `target`.  The histogram of
// all tokens over the steps of z is in shared memory; a bin that has to be
// refined overwrites it (*stale).
template <bool BY_COUNT>
__device__ Cut find_cut(cg::cluster_group& cl, Shared& sh, const Segment& seg, const Row& row,
                        u64 target, bool* stale) {
  const int rank = (int)cl.block_rank();
  Found f = find_bin<BY_COUNT>(cl, sh, target);
  const int zbin = f.bin;
  u64 before_w = f.before_w;  // mass before the bin (0 if masses are not kept)
  u64 left = target - (BY_COUNT ? (u64)f.before_c : f.before_w);  // to reach inside the bin
  uint32_t members = f.bin_c;
  // refinement by the bits of the order key: 11, 11, 10 from the top, larger
  // keys in lower bins
  int sh_bits = 32;
  uint32_t prefix = 0;
  while (members > SM_CAND && sh_bits > 0) {
    const int bits = sh_bits == 10 ? 10 : 11, down = sh_bits - bits, up = sh_bits;
    const uint32_t pre = prefix;
    histogram<true, true>(cl, sh, seg, row, [&](float l) {
      const uint32_t k = max_key(l);
      if ((up < 32 && (k >> up) != pre) || row.bin(l) != zbin) return -1;
      return (SM_BINS - 1) - (int)((k >> down) & ((1u << bits) - 1u));
    });
    *stale = true;
    f = find_bin<BY_COUNT>(cl, sh, left);
    before_w += f.before_w;
    left -= BY_COUNT ? (u64)f.before_c : f.before_w;
    prefix = (up < 32 ? prefix << bits : 0u) | (uint32_t)((SM_BINS - 1) - f.bin);
    sh_bits = down;
    members = f.bin_c;
  }
  Cut cut;
  if (members > SM_CAND) {  // all of one logit: the n-th lowest id of them
    const uint32_t key = prefix;
    const u64 w = row.weight(key_value(key));
    const u64 nth = BY_COUNT ? left : (left + w - 1) / w;
    u64 all;
    cut.id = ordered_pick(
        cl, sh, seg, [&](float l, int) { return (u64)(max_key(l) == key ? 1 : 0); },
        [&](u64) { return nth; }, &all);
    cut.key = key;
    cut.mass = before_w + nth * w;
    return cut;
  }
  // collect the bin's tokens in rank 0 and rank them against one another
  Shared& zero = *cl.map_shared_rank(&sh, 0);
  if (rank == 0 && threadIdx.x == 0) sh.n_cand = 0;
  cl.sync();
  for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) {
    const float l = seg.at(i);
    const uint32_t k = max_key(l);
    if ((sh_bits < 32 && (k >> sh_bits) != prefix) || row.bin(l) != zbin) continue;
    const uint32_t at = atomicAdd(&zero.n_cand, 1u);
    if (at < SM_CAND) {
      zero.cand[at].key = k;
      zero.cand[at].id = seg.id0 + i;
      zero.cand[at].w = row.weight(l);
    }
  }
  cl.sync();
  if (rank == 0) {
    const int m = (int)min(sh.n_cand, (uint32_t)SM_CAND);
    for (int a = threadIdx.x; a < m; a += SM_THREADS) {
      const Cand me = sh.cand[a];
      u64 sum_w = 0;
      uint32_t sum_c = 0;
      for (int b = 0; b < m; b++) {
        const Cand o = sh.cand[b];
        if (o.key > me.key || (o.key == me.key && o.id < me.id)) {
          sum_w += o.w;
          sum_c++;
        }
      }
      const u64 lo = BY_COUNT ? (u64)sum_c : sum_w, step = BY_COUNT ? 1ull : me.w;
      if (lo < left && left <= lo + step) {
        for (int r = 0; r < (int)cl.num_blocks(); r++) {
          Shared& o = *cl.map_shared_rank(&sh, r);
          o.cut_key = me.key;
          o.cut_id = me.id;
          o.cut_w = before_w + sum_w + me.w;
        }
      }
    }
  }
  cl.sync();
  cut.key = sh.cut_key;
  cut.id = sh.cut_id;
  cut.mass = sh.cut_w;
  return cut;
}

__global__ void __launch_bounds__(SM_THREADS, 1)
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

  // ---- the segment into shared memory; its largest logit, NaN and +inf
  float mx = -INFINITY;
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
    for (int i = threadIdx.x; i < n4; i += SM_THREADS * 4) {
      float4 t[4];
#pragma unroll
      for (int v = 0; v < 4; v++)
        if (i + v * SM_THREADS < n4) t[v] = __ldcs(g4 + i + v * SM_THREADS);
#pragma unroll
      for (int v = 0; v < 4; v++)
        if (i + v * SM_THREADS < n4) {
          reinterpret_cast<float4*>(buf)[i + v * SM_THREADS] = t[v];
          see(t[v].x), see(t[v].y), see(t[v].z), see(t[v].w);
        }
    }
    for (int i = 4 * n4 + threadIdx.x; i < seg.cap; i += SM_THREADS) see(buf[i] = seg.g[i]);
  } else {
    for (int i = threadIdx.x; i < seg.cap; i += SM_THREADS) see(buf[i] = seg.g[i]);
  }
  for (int i = seg.cap + threadIdx.x; i < seg.len; i += SM_THREADS) see(seg.g[i]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  if ((threadIdx.x & 31) == 0) sh.part32[threadIdx.x >> 5] = max_key(mx);
  const int any_nan = __syncthreads_or(nan);
  u64 fin;
  block_prefix(finite, sh, &fin);
  if (threadIdx.x == 0) {
    uint32_t key = 0;
    for (int w = 0; w < SM_WARPS; w++) key = max(key, sh.part32[w]);
    sh.pub_key = key;
    sh.pub_bad = any_nan;
    sh.pub_c = (uint32_t)fin;
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
  row.cut_key = 0x00800000u;  // the key of -FLT_MAX
  row.cut_id = a.V;
  row.min_w = (u64)floor((double)min_p * 4294967296.0);
  const u64 P = (u64)floor((double)top_p * 4294967296.0);
  const bool by_k = k > 0 && (uint32_t)k < n_fin, by_p = P < (1ull << 32);
  if (by_k || by_p) {
    const auto zbin = [&](float l) { return row.bin(l); };
    bool stale = false;
    if (by_p)
      histogram<true, true>(cl, sh, seg, row, zbin);
    else
      histogram<true, false>(cl, sh, seg, row, zbin);
    u64 S = 0;
    if (by_k) {
      const Cut c = find_cut<true>(cl, sh, seg, row, (u64)k, &stale);
      row.cut_key = c.key;
      row.cut_id = c.id;
      S = c.mass;
    }
    if (by_p) {
      if (stale) histogram<true, true>(cl, sh, seg, row, zbin);
      if (!by_k)
        for (int q = 0; q < n; q++) S += *cl.map_shared_rank(&sh.pub_w, q);
      // the first token at which the mass reaches ceil(P S / 2^32)
      const u128 prod = (u128)P * S;
      u64 need = (u64)((prod + 0xFFFFFFFFull) >> 32);
      if (need == 0) need = 1;
      const Cut c = find_cut<false>(cl, sh, seg, row, need, &stale);
      row.cut_key = c.key;
      row.cut_id = c.id;
    }
  }

  // ---- the draw, in the order of ids
  const uint32_t u = a.u[r];
  u64 total;
  const int tok = ordered_pick(
      cl, sh, seg,
      [&](float l, int id) {
        if (!row.inside(l, id)) return 0ull;
        const u64 w = row.weight(l);
        return w >= row.min_w ? w : 0ull;
      },
      [&](u64 all) { return (u64)scaled_threshold(u, all) + 1; }, &total);
  if (rank == 0 && threadIdx.x == 0) a.token[r] = tok;
  if (a.n_kept == nullptr && frow == nullptr) return;
  int kept = 0;
  for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) {
    const float l = seg.at(i);
    const bool in = row.inside(l, seg.id0 + i) && (row.min_w == 0 || row.weight(l) >= row.min_w);
    kept += in;
    if (frow != nullptr) frow[i] = in ? l : SPEC_FILTERED;
  }
  if (a.n_kept != nullptr) {
    u64 cta;
    block_prefix(kept, sh, &cta);
    if (threadIdx.x == 0) sh.pub_c = (uint32_t)cta;
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
  int cl = 1;
  while (cl < SM_MAX_CL && V > 4096 * cl) cl *= 2;
  a.seg = ((V + cl - 1) / cl + 3) / 4 * 4;
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
