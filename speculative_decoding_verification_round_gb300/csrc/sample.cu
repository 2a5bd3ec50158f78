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
//  - top-k: every four threads know the largest of the logits that they loaded;
//    the k-th largest of these is a bound that at least k tokens, and
//    typically few more, reach.  Those are collected in every CTA, which all
//    find the cut among them: nobody has to be asked.
//  - top-p alone: a histogram of masses over equal steps of z gives the step
//    that holds the cut; its tokens are collected.
//  - a step with too many tokens (or a top-k whose bound is reached by too
//    many) is refined by the bits of the order key, down to tokens of equal
//    logits, whose cut is the n-th lowest id.
//
// Bound by latency: one row of 151936 logits (0.6 MB) takes 11 us without
// filters, 21 with a top-k, 23 with all filters, 28 with a top-p alone: the
// load, then six to ten meetings of the cluster or the CTA at 0.6 to 1.5 us.
// Many long rows, for which these would add up, go in passes (sample_rows.cu).
#include <cooperative_groups.h>

#include <algorithm>

#include "sample.cuh"

namespace cg = cooperative_groups;

namespace {

struct alignas(16) Shared : ListSmem {  // the row's logits (16-byte stores) follow it
  union {
    struct {  // until the tokens are collected
      u64 slice_w[SM_BINS];  // this rank's share of the combined bins: inclusive sums
      uint32_t slice_c[SM_BINS];
    };
    struct {
      u64 key[SM_CAND];     // the row's collected tokens
      uint32_t w[SM_CAND];  // their weights, 2^32 as 2^32 - 1 (which no other weight is)
    };
  };
  float warp_max[SM_WARPS];
  float cta_max;  // published at the start, with the groups'
  uint32_t own_group[SM_GROUPS];
  u64 pub_w;  // this rank's published totals of the bins, and of the draw
  uint32_t pub_c;
  u64 draw_w;
  uint32_t draw_c;
  uint32_t n_own;
  // published by the rank that finds it: two, in turn, so that one may be
  // written while the other is read
  struct {
    int bin;
    u64 before_w;
    uint32_t before_c, bin_c;
  } found[2];
  int pick;
};
static_assert(sizeof(Shared) % 16 == 0, "the logits behind it are 16-byte aligned");

// The ranks' values at *p: their sum, and the sum of those in front of this
// rank; a lane reads a rank's, so that the remote loads are in flight together.
template <class T>
__device__ __forceinline__ T over_ranks(cg::cluster_group& cl, T* p, T* before) {
  const int lane = threadIdx.x & 31, rank = (int)cl.block_rank();
  T v = lane < (int)cl.num_blocks() ? *cl.map_shared_rank(p, lane) : T(0), front = lane < rank ? v : T(0);
#pragma unroll
  for (int off = SM_MAX_CL / 2; off > 0; off >>= 1) {
    v += __shfl_xor_sync(0xffffffffu, v, off);
    front += __shfl_xor_sync(0xffffffffu, front, off);
  }
  *before = __shfl_sync(0xffffffffu, front, 0);
  return __shfl_sync(0xffffffffu, v, 0);
}

// The row's segment of this CTA.
struct Segment {
  const float* s;  // shared memory: the first `cap` logits
  const float* g;  // global memory
  int len, cap, id0;
  __device__ __forceinline__ float at(int i) const { return i < cap ? s[i] : __ldcg(g + i); }
};

// The first id, in the order of ids over the whole row, at which the running
// sum of the weights of measure(two logits, id of the first, count) reaches
// target(total); every thread of the cluster gets it, and the total.  -1 if
// it is never reached.  `count` is summed up as well, for rank 0's *counted.
template <class M, class Tg>
__device__ int ordered_pick(cg::cluster_group& cl, Shared& sh, const Segment& seg, M&& measure,
                            Tg&& target, uint32_t* counted) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  // a thread owns a run of ids; an odd number of pairs keeps its strided
  // reads of shared memory at two wavefronts
  const int c = 2 * (((seg.len + 2 * SM_THREADS - 1) / (2 * SM_THREADS)) | 1);
  const int i0 = min(seg.len, (int)threadIdx.x * c), i1 = min(seg.len, i0 + c);
  auto pair = [&](int i) {  // the second of the last pair may be past the end
    if (i + 1 < i1) return i + 1 < seg.cap ? *reinterpret_cast<const float2*>(seg.s + i) : make_float2(seg.at(i), seg.at(i + 1));
    return make_float2(seg.at(i), -INFINITY);
  };
  u64 mine = 0;
  uint32_t cnt = 0;
  for (int i = i0; i < i1; i += 2) {
    const uint2 w = measure(pair(i), seg.id0 + i, cnt);
    mine += w.x;
    mine += w.y;
    mine += (w.x == 0xFFFFFFFFu) + (w.y == 0xFFFFFFFFu);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, off);
  if ((threadIdx.x & 31) == 0) sh.part32[threadIdx.x >> 5] = cnt;
  u64 cta;
  const u64 incl = block_prefix(mine, sh, &cta);
  if (threadIdx.x == 0) {
    uint32_t all = 0;
    for (int w = 0; w < SM_WARPS; w++) all += sh.part32[w];
    sh.draw_w = cta;
    sh.draw_c = all;
    sh.pick = -1;
  }
  cl.sync();
  u64 before;
  const u64 all = over_ranks(cl, &sh.draw_w, &before);
  if (counted != nullptr && rank == 0 && threadIdx.x < 32) {
    uint32_t front;
    *counted = over_ranks(cl, &sh.draw_c, &front);
  }
  const u64 t = target(all);
  const u64 hi = before + incl, lo = hi - mine;
  // at most one thread's run holds it; its warp goes through the run, a lane a pair
  const unsigned owner = __ballot_sync(0xffffffffu, mine > 0 && lo < t && t <= hi);
  if (owner != 0u) {
    const int lane = threadIdx.x & 31, who = __ffs(owner) - 1;
    const int j0 = __shfl_sync(0xffffffffu, i0, who), j1 = __shfl_sync(0xffffffffu, i1, who);
    u64 run = __shfl_sync(0xffffffffu, lo, who);
    for (int base = j0; base < j1; base += 64) {
      const int i = base + 2 * lane;
      uint2 w = make_uint2(0u, 0u);
      if (i < j1) w = measure(make_float2(seg.at(i), i + 1 < j1 ? seg.at(i + 1) : -INFINITY), seg.id0 + i, cnt);
      const u64 wx = widen(w.x), both = wx + widen(w.y);
      u64 upto = both;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run + upto >= t);
      if (hit != 0u) {
        const int first = __ffs(hit) - 1;
        const int id = __shfl_sync(0xffffffffu, seg.id0 + i + (run + upto - both + wx >= t ? 0 : 1), first);
        if (lane < n) *cl.map_shared_rank(&sh.pick, lane) = id;
        break;
      }
      run += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  cl.sync();
  return sh.pick;
}

// The combined bins of the cluster from every CTA's: every rank holds its
// share of them as inclusive sums.
template <bool COUNT, bool MASS>
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
#pragma unroll 8
      for (int r = 0; r < n; r++) {
        if (COUNT) cc[k] += cl.map_shared_rank(sh.cnt, r)[b0 + b];
        if (MASS)
          w[k] += ((u64)cl.map_shared_rank(sh.hi, r)[b0 + b] << 16) + cl.map_shared_rank(sh.lo, r)[b0 + b];
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

__device__ __forceinline__ void clear_bins(Shared& sh) {
  for (int b = threadIdx.x; b < 3 * SM_BINS; b += SM_THREADS) sh.cnt[b] = 0;  // cnt, lo, hi
  __syncthreads();
}
// Histogram of all tokens over the steps of z (two 32-bit additions a mass:
// 64-bit ones in shared memory are compare-and-swap loops, 24 us for a CTA's
// 30720 logits where these take 3).
template <bool COUNT>
__device__ void histogram(cg::cluster_group& cl, Shared& sh, const Segment& seg, const Row& row) {
  clear_bins(sh);
  for (int i = 2 * threadIdx.x; i < seg.len; i += 2 * SM_THREADS) {
    const bool two = i + 1 < seg.len;
    const float2 x = row.x2(make_float2(seg.at(i), two ? seg.at(i + 1) : -INFINITY));
    const uint2 w = Row::w2(x);
    const int b0 = Row::bin_of(x.x), b1 = Row::bin_of(x.y);
    if (COUNT) atomicAdd(&sh.cnt[b0], 1u);
    if (COUNT && two) atomicAdd(&sh.cnt[b1], 1u);
    if (w.x != 0) add_mass(sh, b0, w.x);
    if (w.y != 0) add_mass(sh, b1, w.y);
  }
  combine<COUNT, true>(cl, sh);
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
__device__ Found find_bin(cg::cluster_group& cl, Shared& sh, u64 target, int& turn) {
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  const int share = SM_BINS / n;
  u64 bw;
  uint32_t bc;
  over_ranks(cl, &sh.pub_w, &bw);
  over_ranks(cl, &sh.pub_c, &bc);
  const u64 base = BY_COUNT ? bc : bw;
  for (int b = threadIdx.x; b < share; b += SM_THREADS) {
    const u64 hi = base + (BY_COUNT ? (u64)sh.slice_c[b] : sh.slice_w[b]);
    const u64 lo = base + (b == 0 ? 0ull : BY_COUNT ? (u64)sh.slice_c[b - 1] : sh.slice_w[b - 1]);
    if (lo < target && target <= hi) {
      const u64 pw = b == 0 ? 0ull : sh.slice_w[b - 1];
      const uint32_t pc = b == 0 ? 0u : sh.slice_c[b - 1];
      for (int r = 0; r < n; r++) {
        auto& o = cl.map_shared_rank(&sh, r)->found[turn];
        o.bin = rank * share + b;
        o.before_w = bw + pw;
        o.before_c = bc + pc;
        o.bin_c = sh.slice_c[b] - pc;
      }
    }
  }
  cl.sync();
  Found f;
  f.bin = sh.found[turn].bin;
  f.before_w = sh.found[turn].before_w;
  f.before_c = sh.found[turn].before_c;
  f.bin_c = sh.found[turn].bin_c;
  turn ^= 1;
  return f;
}

// The tokens that take(logit) accepts, collected into every CTA's sh.key and
// sh.w; returns their number, or more than SM_CAND if they are too many.
template <class P>
__device__ int collect(cg::cluster_group& cl, Shared& sh, const Segment& seg, const Row& row, bool mass,
                       P&& take) {
  const int n = (int)cl.num_blocks();
  if (threadIdx.x == 0) sh.n_own = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) {
    const float l = seg.at(i);
    if (take(l)) {
      const uint32_t at = atomicAdd(&sh.n_own, 1u);
      if (at < SM_LOCAL) {
        sh.own_key[at] = Row::composite(max_key(l), seg.id0 + i);
      }
    }
  }
  cl.sync();  // (and the combined bins have been read, which the tokens now overwrite)
  uint32_t before;
  const uint32_t all = over_ranks(cl, &sh.n_own, &before);
  const int lane = threadIdx.x & 31;
  const bool over = __any_sync(0xffffffffu, lane < n && *cl.map_shared_rank(&sh.n_own, min(lane, n - 1)) > SM_LOCAL);
  if (!over && all <= SM_CAND) {
    // a thread has a token and a part of the ranks
    const int own = (int)sh.n_own;
    int parts = 1;
    while (parts < n && own * parts * 2 <= SM_THREADS) parts *= 2;
    for (int e = threadIdx.x; e < own * parts; e += SM_THREADS) {
      const int c = e / parts;
      const u64 key = sh.own_key[c];
      const uint32_t w = mass ? row.weight(key_value((uint32_t)(key >> 20))) : 0u;
      for (int r = e % parts; r < n; r += parts) {
        Shared& o = *cl.map_shared_rank(&sh, r);
        o.key[before + c] = key;
        o.w[before + c] = w;
      }
    }
  }
  cl.sync();
  return over ? SM_CAND + 1 : (int)all;
}

// The token at which the running sum of counts (BY_COUNT) or masses, in the
// order (logit descending, id ascending), reaches `target`.  The histogram of
// all tokens over the steps of z is combined; the search overwrites it.
template <bool BY_COUNT>
__device__ Cut find_cut(cg::cluster_group& cl, Shared& sh, const Segment& seg, const Row& row,
                        u64 target, int& turn) {
  Found f = find_bin<BY_COUNT>(cl, sh, target, turn);
  const int zbin = f.bin;
  u64 before_w = f.before_w;
  u64 left = target - (BY_COUNT ? (u64)f.before_c : f.before_w);  // to reach inside the bin
  // refinement by the bits of the order key: 10, 10, 10, 2 from the top,
  // larger keys in lower bins
  int known = 32;  // bits still unknown
  uint32_t prefix = 0;
  auto member = [&](float l, uint32_t k) {
    return (known >= 32 || (k >> known) == prefix) && row.bin(l) == zbin;
  };
  int m = SM_CAND + 1;
  for (;;) {
    if (!BY_COUNT || f.bin_c <= SM_CAND)
      m = collect(cl, sh, seg, row, true, [&](float l) { return member(l, max_key(l)); });
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
    combine<true, true>(cl, sh);
    f = find_bin<BY_COUNT>(cl, sh, left, turn);
    before_w += f.before_w;
    left -= BY_COUNT ? (u64)f.before_c : f.before_w;
    prefix = (known < 32 ? prefix << bits : 0u) | (uint32_t)((SM_BINS - 1) - f.bin);
    known = down;
  }
  Cut cut;
  if (m > SM_CAND) {  // all of one logit: the n-th lowest id of them
    const uint32_t key = prefix;
    const u64 w = widen(row.weight(key_value(key)));
    const u64 nth = BY_COUNT ? left : (left + w - 1) / w;
    const int id = ordered_pick(
        cl, sh, seg,
        [&](float2 l, int, uint32_t&) { return make_uint2(max_key(l.x) == key, max_key(l.y) == key); },
        [&](u64) { return nth; }, nullptr);
    cut.key = Row::composite(key, id);
    cut.mass = before_w + nth * w;
    return cut;
  }
  cut = cut_list(sh, sh.key, sh.w, m, BY_COUNT, true, left, 20 + known, known >= 32 ? 0u : prefix);
  cut.mass += before_w;
  return cut;
}

// One row by its cluster.
__device__ __forceinline__ void sample_row(const SampleArgs& a, cg::cluster_group& cl, Shared& sh, float* buf,
                                           int r) {
  const int n = (int)cl.num_blocks(), rank = (int)cl.block_rank();
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

  // ---- the segment into shared memory; its largest logit (NaN if there is one)
  float mx = -INFINITY;  // of this thread's
  auto see = [&](float l) { asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx) : "f"(l)); };
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
  float gmx = mx, wmx;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, off == 4 ? gmx : off > 4 ? wmx : gmx, off);
    if (off < 4) {
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(gmx) : "f"(o));
    } else {
      if (off == 4) wmx = gmx;
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(wmx) : "f"(o));
    }
  }
  if ((threadIdx.x & 3) == 0) sh.own_group[threadIdx.x >> 2] = max_key(gmx);
  if ((threadIdx.x & 31) == 0) sh.warp_max[threadIdx.x >> 5] = wmx;
  __syncthreads();
  if (threadIdx.x < 32) {
    wmx = threadIdx.x < SM_WARPS ? sh.warp_max[threadIdx.x] : -INFINITY;
#pragma unroll
    for (int off = SM_WARPS / 2; off > 0; off >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, wmx, off);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(wmx) : "f"(o));
    }
    if (threadIdx.x == 0) sh.cta_max = wmx;
  }
  cl.sync();
  float top = (int)(threadIdx.x & 31) < n ? *cl.map_shared_rank(&sh.cta_max, threadIdx.x & 31) : -INFINITY;
#pragma unroll
  for (int off = SM_MAX_CL / 2; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, top, off);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(o));
  }
  top = __shfl_sync(0xffffffffu, top, 0);
  row.zmax = row_zmax(max_key(top), row.T);
  row.plain |= Row::far(row.zmax);
  bad |= !(fabsf(top) < INFINITY) || !(fabsf(row.zmax) < INFINITY);  // NaN, +inf, nothing but -inf
  float* frow = a.filtered != nullptr ? a.filtered + (int64_t)r * a.ldf + seg.id0 : nullptr;
  if (bad) {  // the whole cluster
    if (frow != nullptr)
      for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) frow[i] = __int_as_float(0x7FFFFFFF);
    if (rank == 0 && threadIdx.x == 0) {
      a.token[r] = -1;
      if (a.n_kept != nullptr) a.n_kept[r] = 0;
    }
    cl.sync();  // shared memory stays until everybody has read it
    return;
  }

  // ---- the cuts.  Everything above -inf is inside at first.
  row.no_cut();
  const u64 M = (u64)floor((double)min_p * 4294967296.0);
  row.min_w = (uint32_t)min(M, 0xFFFFFFFFull);
  const u64 P = (u64)floor((double)top_p * 4294967296.0);
  const bool by_k = k > 0 && k < a.V, by_p = P < (1ull << 32);
  int turn = 0;
  bool done = false;
  if (by_k) {
    // a bound that at least k tokens reach, and hardly more than SM_CAND
    const int groups = n * SM_GROUPS;
    float bound = -INFINITY;
    int bin = -1;
    if (k <= groups * 3 / 4) {
      // the k-th largest of the groups' largest, bit by bit (its order key's
      // first 20: a bound may be a little low)
      constexpr int PER = SM_MAX_CL * SM_GROUPS / SM_THREADS;
      uint32_t mine[PER];
#pragma unroll
      for (int e = 0; e < PER; e++) {
        const int g = (int)threadIdx.x + e * SM_THREADS;
        mine[e] = g < groups ? cl.map_shared_rank(sh.own_group, g / SM_GROUPS)[g % SM_GROUPS] : 0u;
      }
      uint32_t low = 0u;
      for (int bit = 30; bit >= 12; bit -= 2) {
        uint32_t c12 = 0, c3 = 0;  // at least low + 1, 2, 3 steps
#pragma unroll
        for (int e = 0; e < PER; e++) {
          c12 += mine[e] >= (low | (1u << bit)) ? 1u : 0u;
          c12 += mine[e] >= (low | (2u << bit)) ? 1u << 16 : 0u;
          c3 += mine[e] >= (low | (3u << bit)) ? 1u : 0u;
        }
        c12 = __reduce_add_sync(0xffffffffu, c12);
        c3 = __reduce_add_sync(0xffffffffu, c3);
        uint32_t* part = sh.part32 + (bit & 2) * SM_WARPS;  // two, in turn: one barrier a step
        if ((threadIdx.x & 31) == 0) {
          part[threadIdx.x >> 5] = c12;
          part[SM_WARPS + (threadIdx.x >> 5)] = c3;
        }
        __syncthreads();
        const int lane = threadIdx.x & 31;
        c12 = __reduce_add_sync(0xffffffffu, lane < SM_WARPS ? part[lane] : 0u);
        c3 = __reduce_add_sync(0xffffffffu, lane < SM_WARPS ? part[SM_WARPS + lane] : 0u);
        const uint32_t step = c3 >= (uint32_t)k ? 3u : (c12 >> 16) >= (uint32_t)k ? 2u : (c12 & 0xFFFFu) >= (uint32_t)k ? 1u : 0u;
        low |= step << bit;
      }
      // -inf or below: fewer than k groups have a finite logit
      if (low > 0x007FFFFFu) bound = key_value(low);
    } else if (k <= SM_CAND) {  // to a step of z: the k-th largest of all tokens
      clear_bins(sh);
      for (int i = 2 * threadIdx.x; i < seg.len; i += 2 * SM_THREADS) {
        const bool two = i + 1 < seg.len;
        const float2 x = row.x2(make_float2(seg.at(i), two ? seg.at(i + 1) : -INFINITY));
        atomicAdd(&sh.cnt[Row::bin_of(x.x)], 1u);
        if (two) atomicAdd(&sh.cnt[Row::bin_of(x.y)], 1u);
      }
      combine<true, false>(cl, sh);
      bin = find_bin<true>(cl, sh, (u64)k, turn).bin;
    }
    int m = SM_CAND + 1;
    if (bound > -INFINITY)
      m = collect(cl, sh, seg, row, by_p, [&](float l) { return l >= bound; });
    else if (bin >= 0)
      m = collect(cl, sh, seg, row, by_p, [&](float l) { return row.bin(l) <= bin; });
    if (m <= SM_CAND) {
      // the keys agree above the first bit in which the bound and the largest differ
      int open = 32;
      u64 prefix = 0;
      if (bound > -INFINITY) {
        const uint32_t hi = max_key(top), lo = max_key(bound);
        open = 32 - __clz(hi ^ lo);
        prefix = open < 32 ? hi >> open : 0u;
      }
      Cut c = cut_list(sh, sh.key, sh.w, m, true, by_p, (u64)k, 20 + open, prefix);
      if (by_p) c = cut_list(sh, sh.key, sh.w, m, false, true, mass_needed(P, c.mass), 20 + open, prefix);
      row.set_cut(c.key);
      done = true;
    }
  }
  if (!done && (by_k || by_p)) {
    u64 S = 0;
    if (by_k) {
      histogram<true>(cl, sh, seg, row);
      const Cut c = find_cut<true>(cl, sh, seg, row, (u64)k, turn);
      row.set_cut(c.key);
      S = c.mass;
    }
    if (by_p) {
      histogram<false>(cl, sh, seg, row);
      u64 front;
      if (!by_k) S = over_ranks(cl, &sh.pub_w, &front);
      row.set_cut(find_cut<false>(cl, sh, seg, row, mass_needed(P, S), turn).key);
    }
  }

  // ---- the draw, in the order of ids
  const uint32_t u = a.u[r];
  uint32_t kept = 0;
  const int tok = ordered_pick(
      cl, sh, seg,
      [&](float2 l, int id, uint32_t& cnt) {
        uint2 w = make_uint2(0u, 0u);
        if (l.x >= row.least || l.y >= row.least) {
          w = row.weight2(l);
          const bool in_x = row.inside(l.x, id) && w.x >= row.min_w;
          const bool in_y = row.inside(l.y, id + 1) && w.y >= row.min_w;
          cnt += in_x;
          cnt += in_y;
          w.x = in_x ? w.x : 0u;
          w.y = in_y ? w.y : 0u;
        }
        return w;
      },
      [&](u64 all) { return (u64)scaled_threshold(u, all) + 1; }, &kept);
  if (rank == 0 && threadIdx.x == 0) {
    a.token[r] = tok;
    if (a.n_kept != nullptr) a.n_kept[r] = (int)kept;
  }
  if (frow == nullptr) return;
  auto out = [&](float l, int id) {
    const bool in = row.inside(l, id) && (row.min_w == 0u || row.weight(l) >= row.min_w);
    return in ? l : SPEC_FILTERED;
  };
  if ((reinterpret_cast<uintptr_t>(frow) & 15u) == 0 && seg.cap == seg.len) {
    const int n4 = seg.len / 4;
    for (int i = threadIdx.x; i < n4; i += SM_THREADS) {
      const float4 l = reinterpret_cast<const float4*>(buf)[i];
      const int id = seg.id0 + 4 * i;
      __stcs(reinterpret_cast<float4*>(frow) + i,
             make_float4(out(l.x, id), out(l.y, id + 1), out(l.z, id + 2), out(l.w, id + 3)));
    }
    for (int i = 4 * n4 + threadIdx.x; i < seg.len; i += SM_THREADS) frow[i] = out(buf[i], seg.id0 + i);
  } else {
    for (int i = threadIdx.x; i < seg.len; i += SM_THREADS) frow[i] = out(seg.at(i), seg.id0 + i);
  }
}

template <bool LIST>
__global__ void __launch_bounds__(SM_THREADS, 2)
sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  Shared& sh = *reinterpret_cast<Shared*>(dyn);
  float* buf = reinterpret_cast<float*>(dyn + sizeof(Shared));
  cg::cluster_group cl = cg::this_cluster();
  grid_dep_begin();
  if constexpr (LIST) {
    const int n = (int)cl.num_blocks(), count = *a.n_rows;
    for (int at = blockIdx.x / n; at < count; at += gridDim.x / n) {
      sample_row(a, cl, sh, buf, a.rows[at]);
      cl.sync();  // no CTA reads the row's memory any more
    }
  } else {
    sample_row(a, cl, sh, buf, blockIdx.x / (int)cl.num_blocks());
  }
}

}  // namespace

void sample_init_attrs() {
  sample_rows_init_attrs();
  int dev = 0, optin = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  for (auto kernel : {sample_kernel<false>, sample_kernel<true>}) {
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
    cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  }
}

int sample_clusters_launch(SampleArgs a, int clusters, cudaStream_t st) {
  // CTAs of a row: with 8192 logits each (16384 where the rows alone fill the
  // SMs) a row's CTAs leave room for another cluster's beside them, whose
  // loads go on while these compute
  int cl = 1;
  const int each = (long long)clusters * SM_MAX_CL > 1024 ? 16384 : 4096;
  while (cl < SM_MAX_CL && a.V > each * cl) cl *= 2;
  a.seg = ((a.V + cl - 1) / cl + 3) / 4 * 4;
  if (a.seg > SM_SEG) return fail(SPEC_E_SHAPE, "V above 1048512 is not supported");
  const int room = (int)((227 * 1024 - sizeof(Shared)) / sizeof(float)) / 4 * 4;
  a.cap = std::min(a.seg, room);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cl;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = programmatic_launch() ? 2 : 1;
  cfg.gridDim = dim3((unsigned)clusters * cl);
  cfg.blockDim = dim3(SM_THREADS);
  cfg.dynamicSmemBytes = sizeof(Shared) + sizeof(float) * (size_t)a.cap;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, a.rows != nullptr ? sample_kernel<true> : sample_kernel<false>, a);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("sample: ") + cudaGetErrorString(e));
  return SPEC_OK;
}

// Many long rows go through the passes of sample_rows.cu: 8 rows of 248320
// logits take 35 us in clusters and 37 in passes (of mixed settings; a top-k
// alone 26 and 22), 32 rows 86 and 51; 128 rows of 32000 38 and 47, 256 rows 64
// and 56.
static bool by_passes(int R, int V) {
  return V > 16384 && (long long)R * V > (V > 65536 ? 2000000 : 5000000);
}

size_t sample_bytes(int R, int V) { return by_passes(R, V) ? sample_rows_bytes(R, V) : 0; }

int launch_sample(const float* logits, int R, int V, int64_t ld, const uint32_t* u,
                  const float* temperature, const int32_t* top_k, const float* top_p,
                  const float* min_p, int32_t* token, int32_t* n_kept, float* filtered, int64_t ldf,
                  void* workspace, cudaStream_t st) {
  SampleArgs a = {};
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
  a.R = R;
  a.V = V;
  if (by_passes(R, V)) return sample_rows_launch(a, workspace, st);
  return sample_clusters_launch(a, R, st);
}
