// sample_rows.cu -- filtered sampling of many long rows: passes over all of
// them (the same rules and integer sums as sample.cu, which keeps a row in the
// shared memory of a cluster and is bound by its barriers, not by the memory,
// once rows are many).
//
// A row is one of three kinds, by its settings: top-k (with or without the
// other filters), top-p alone, or neither.  Streaming passes have a CTA per
// 8192 logits of a row, a warp per 1024 of them; between them a CTA per row
// decides.
//   maxima   stream: the largest logit of every 128
//   bound    row: the largest, the settings, and for a top-k a bound that at
//            least k of the groups of 128 reach
//   pass     stream: top-k rows collect the tokens at the bound; top-p rows
//            add their masses up over steps of z; the others over 1024 ids
//   cut      row: top-k rows find their cut among the collected tokens and
//            draw from them; rows without filters draw; top-p rows find the
//            step that holds their cut
//   step     stream, top-p rows: the masses above that step over 1024 ids,
//            its tokens collected
//   draw     row, top-p rows: the cut, and the draw
//   filter   stream, where filtered logits are wanted
// A row that collects too many tokens goes to the clusters of sample.cu as a
// whole.  Each kernel is a programmatic dependent of the one in front of it.
#include <algorithm>

#include "sample.cuh"

namespace {

constexpr int SR_GROUP = 128;   // logits whose largest is kept
constexpr int SR_RANGE = 1024;  // logits of a warp, and ids whose mass is kept
constexpr int SR_WARPS = 8;
constexpr int SR_THREADS = 32 * SR_WARPS;
constexpr int SR_SEG = SR_RANGE * SR_WARPS;
constexpr int SR_LIST = 8192;   // tokens that are collected of a row
constexpr int SR_MAX_K = 2048;  // of a top-k by a bound, so that these are enough mostly
constexpr int SR_MAX_RANGES = 1024;
constexpr int SR_HARD_CLUSTERS = 16;

enum RowKind : int { ROW_BAD, ROW_PLAIN, ROW_TOP_K, ROW_TOP_P, ROW_HARD };

struct RowState {
  Row row;  // least, last_id: the cut, once `done`
  float top, bound;
  int kind, k;
  u64 P;
  u64 left;  // top-p: the mass to reach inside the step
  int bin;
  uint32_t listed;
};

// One row's workspace.
struct RowSpace {
  RowState* state;
  uint32_t* group;  // order keys
  u64* mass;        // top-p: over SM_BINS steps of z
  u64* key;         // collected tokens
  uint32_t* w;
  u64* range_w;  // over SR_RANGE ids
  uint32_t* range_c;
};

struct Spaces {
  char* base;
  int32_t* hard;  // rows for the clusters, and their number in front
  size_t stride;  // bytes of a row
  int groups, ranges;
  __host__ __device__ static size_t up(size_t b) { return (b + 127) / 128 * 128; }
  __host__ __device__ RowSpace row(int r) const {
    RowSpace s;
    char* p = base + stride * r;
    s.state = reinterpret_cast<RowState*>(p);
    p += up(sizeof(RowState));
    s.mass = reinterpret_cast<u64*>(p);
    p += up(sizeof(u64) * SM_BINS);
    s.key = reinterpret_cast<u64*>(p);
    p += up(sizeof(u64) * SR_LIST);
    s.w = reinterpret_cast<uint32_t*>(p);
    p += up(sizeof(uint32_t) * SR_LIST);
    s.range_w = reinterpret_cast<u64*>(p);
    p += up(sizeof(u64) * ranges);
    s.range_c = reinterpret_cast<uint32_t*>(p);
    p += up(sizeof(uint32_t) * ranges);
    s.group = reinterpret_cast<uint32_t*>(p);
    return s;
  }
};

Spaces spaces(void* workspace, int R, int V) {
  Spaces s;
  s.groups = (V + SR_GROUP - 1) / SR_GROUP;
  s.ranges = (V + SR_RANGE - 1) / SR_RANGE;
  s.stride = Spaces::up(sizeof(RowState)) + Spaces::up(sizeof(u64) * SM_BINS) + Spaces::up(sizeof(u64) * SR_LIST) +
             Spaces::up(sizeof(uint32_t) * SR_LIST) + Spaces::up(sizeof(u64) * s.ranges) +
             Spaces::up(sizeof(uint32_t) * s.ranges) + Spaces::up(sizeof(uint32_t) * s.groups);
  s.hard = reinterpret_cast<int32_t*>(workspace);
  s.base = reinterpret_cast<char*>(workspace) + Spaces::up(sizeof(int32_t) * ((size_t)R + 1));
  return s;
}

// Up to four logits of the 128 from id g0 on, for this lane: ids g0 + 4 lane
// .. (16-byte loads) where the row is aligned, else g0 + lane + 32 e.
struct Quad {
  float l[4];
  int id[4];
};
__device__ __forceinline__ Quad load_quad(const float* row, bool aligned, int g0, int V, int lane) {
  Quad q;
  if (aligned && g0 + SR_GROUP <= V) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(row + g0) + lane);
    q.l[0] = v.x, q.l[1] = v.y, q.l[2] = v.z, q.l[3] = v.w;
#pragma unroll
    for (int e = 0; e < 4; e++) q.id[e] = g0 + 4 * lane + e;
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++) {
      q.id[e] = g0 + lane + 32 * e;
      q.l[e] = q.id[e] < V ? __ldcs(row + q.id[e]) : -INFINITY;
    }
  }
  return q;
}

// ---------------------------------------------------------------------------
// maxima
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(SR_THREADS)
sr_maxima_kernel(const SampleArgs a, const Spaces sp, int segs) {
  grid_dep_launch();
  const int r = blockIdx.x / segs, seg = blockIdx.x % segs;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RowSpace s = sp.row(r);
  if (seg == 0) {
    for (int b = threadIdx.x; b < SM_BINS; b += SR_THREADS) s.mass[b] = 0;
    if (threadIdx.x == 0) {
      s.state->listed = 0;
      if (r == 0) sp.hard[0] = 0;
    }
  }
  const float* row = a.logits + (int64_t)r * a.ld;
  const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
  const int v0 = seg * SR_SEG + warp * SR_RANGE;
  constexpr int G = SR_RANGE / SR_GROUP;
  float mx[G];
#pragma unroll
  for (int g = 0; g < G; g++) {
    const Quad q = load_quad(row, aligned, v0 + g * SR_GROUP, a.V, lane);
    float m = q.l[0];
#pragma unroll
    for (int e = 1; e < 4; e++) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(q.l[e]));
    mx[g] = m;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int g = 0; g < G; g++) {
      const float o = __shfl_xor_sync(0xffffffffu, mx[g], off);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx[g]) : "f"(o));
    }
  float mine = mx[0];
#pragma unroll
  for (int g = 1; g < G; g++) mine = lane == g ? mx[g] : mine;
  const int at = v0 / SR_GROUP + lane;
  if (lane < G && at < sp.groups) s.group[at] = max_key(mine);  // NaN is above every key
}

// ---------------------------------------------------------------------------
// bound
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(SR_THREADS)
sr_bound_kernel(const SampleArgs a, const Spaces sp) {
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_part[4][SR_WARPS];
  grid_dep_launch();
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RowSpace s = sp.row(r);
  RowState st = {};
  Row& row = st.row;
  row.T = a.temperature != nullptr ? a.temperature[r] : 1.0f;
  st.k = a.top_k != nullptr ? a.top_k[r] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[r] : 1.0f;
  const float min_p = a.min_p != nullptr ? a.min_p[r] : 0.0f;
  bool bad = !(row.T >= 0.0f && row.T <= FLT_MAX) || st.k < 0 || !(top_p >= 0.0f && top_p <= 1.0f) ||
             !(min_p >= 0.0f && min_p <= 1.0f);
  if (row.T == 0.0f) {  // greedy: the first of the order
    row.T = 1.0f;
    st.k = 1;
  }
  if (bad) row.T = 1.0f;
  row.inv_T = __frcp_rn(row.T);
  row.plain = row.T == 1.0f || !(row.T > 0x1p-60f && row.T < 0x1p60f);
  row.no_cut();
  row.min_w = (uint32_t)min((u64)floor((double)min_p * 4294967296.0), 0xFFFFFFFFull);
  st.P = (u64)floor((double)top_p * 4294967296.0);
  grid_dep_wait();
  uint32_t top = 0;
  for (int g = tid; g < sp.groups; g += SR_THREADS) {
    const uint32_t k = __ldcg(s.group + g);
    s_key[g] = k;
    top = max(top, k);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s_part[0][warp] = top;
  __syncthreads();
  for (int w = 0; w < SR_WARPS; w++) top = max(top, s_part[0][w]);
  __syncthreads();
  const bool finite = top > 0x007FFFFFu && top < 0xFF800000u;  // above -inf, below +inf and NaN
  st.top = finite ? key_value(top) : 0.0f;
  row.zmax = row_zmax(max_key(st.top), row.T);
  bad |= !finite || !(fabsf(row.zmax) < INFINITY);
  const bool by_k = st.k > 0 && st.k < a.V;
  st.bound = -INFINITY;
  st.kind = bad ? ROW_BAD : by_k ? ROW_HARD : st.P < (1ull << 32) ? ROW_TOP_P : ROW_PLAIN;
  if (!bad && by_k && st.k <= SR_MAX_K && st.k <= sp.groups * 3 / 4) {
    // the k-th largest of the groups' largest, two bits a step (the order
    // key's first 20: a bound may be a little low)
    uint32_t low = 0u;
    int turn = 0;
    for (int bit = 30; bit >= 12; bit -= 2) {
      uint32_t c12 = 0, c3 = 0;  // at least low + 1, 2, 3 steps
      for (int g = tid; g < sp.groups; g += SR_THREADS) {
        const uint32_t k = s_key[g];
        c12 += k >= (low | (1u << bit)) ? 1u : 0u;
        c12 += k >= (low | (2u << bit)) ? 1u << 16 : 0u;
        c3 += k >= (low | (3u << bit)) ? 1u : 0u;
      }
      c12 = __reduce_add_sync(0xffffffffu, c12);
      c3 = __reduce_add_sync(0xffffffffu, c3);
      if (lane == 0) {
        s_part[2 * turn][warp] = c12;
        s_part[2 * turn + 1][warp] = c3;
      }
      __syncthreads();
      c12 = __reduce_add_sync(0xffffffffu, lane < SR_WARPS ? s_part[2 * turn][lane] : 0u);
      c3 = __reduce_add_sync(0xffffffffu, lane < SR_WARPS ? s_part[2 * turn + 1][lane] : 0u);
      const uint32_t k = (uint32_t)st.k;
      low |= (c3 >= k ? 3u : (c12 >> 16) >= k ? 2u : (c12 & 0xFFFFu) >= k ? 1u : 0u) << bit;
      turn ^= 1;
    }
    if (low > 0x007FFFFFu) {  // at least k groups have a finite logit
      st.bound = key_value(low);
      st.kind = ROW_TOP_K;
    }
  }
  if (tid == 0) {
    if (bad) {
      a.token[r] = -1;
      if (a.n_kept != nullptr) a.n_kept[r] = 0;
    }
    if (st.kind == ROW_HARD) sp.hard[1 + atomicAdd(sp.hard, 1)] = r;
    *s.state = st;
  }
}

// ---------------------------------------------------------------------------
// pass
// ---------------------------------------------------------------------------
// A CTA's collected tokens (ids of its segment), to the row's list.
struct OwnList {
  u64 key[SM_LOCAL];
  uint32_t n, at;
};
__device__ __forceinline__ void own_add(OwnList& o, float l, int id) {
  const uint32_t at = atomicAdd(&o.n, 1u);
  if (at < SM_LOCAL) o.key[at] = Row::composite(max_key(l), id);
}
__device__ __forceinline__ void own_flush(OwnList& o, const RowSpace& s, const Row& row) {
  __syncthreads();
  const uint32_t n = o.n;
  if (threadIdx.x == 0 && n > 0) o.at = atomicAdd(&s.state->listed, n > SM_LOCAL ? SR_LIST + 1 : n);
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < min(n, (uint32_t)SM_LOCAL); c += SR_THREADS)
    if (o.at + c < SR_LIST) {
      s.key[o.at + c] = o.key[c];
      s.w[o.at + c] = row.weight(key_value((uint32_t)(o.key[c] >> 20)));
    }
}

// Mass and number of the tokens that stay.
struct Sum {
  u64 w = 0;
  uint32_t c = 0;
  __device__ __forceinline__ void add(uint32_t x, bool in) {
    w += in ? x : 0u;
    w += in && x == 0xFFFFFFFFu;
    c += in;
  }
  __device__ __forceinline__ void over_warp() {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
    c = __reduce_add_sync(0xffffffffu, c);
  }
};

__global__ void __launch_bounds__(SR_THREADS)
sr_pass_kernel(const SampleArgs a, const Spaces sp, int segs) {
  __shared__ union {
    struct {
      uint32_t lo[SM_BINS], hi[SM_BINS];
    };
    OwnList own;
  } sh;
  grid_dep_launch();
  const int r = blockIdx.x / segs, seg = blockIdx.x % segs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RowSpace s = sp.row(r);
  const float* lrow = a.logits + (int64_t)r * a.ld;
  const bool aligned = (reinterpret_cast<uintptr_t>(lrow) & 15u) == 0;
  const int v0 = seg * SR_SEG + warp * SR_RANGE;
  constexpr int G = SR_RANGE / SR_GROUP;
  grid_dep_wait();
  const int kind = s.state->kind;
  const Row row = s.state->row;
  if (kind == ROW_TOP_K) {
    const float bound = s.state->bound;
    if (tid == 0) sh.own.n = 0;
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; g++) {
      const Quad q = load_quad(lrow, aligned, v0 + g * SR_GROUP, a.V, lane);
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (q.l[e] >= bound) own_add(sh.own, q.l[e], q.id[e]);
    }
    own_flush(sh.own, s, row);
  } else if (kind == ROW_TOP_P) {
    for (int b = tid; b < SM_BINS; b += SR_THREADS) sh.lo[b] = sh.hi[b] = 0;
    __syncthreads();
#pragma unroll 2
    for (int g = 0; g < G; g++) {
      const Quad q = load_quad(lrow, aligned, v0 + g * SR_GROUP, a.V, lane);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 x = row.x2(make_float2(q.l[e], q.l[e + 1]));
        const uint2 w = Row::w2(x);
        const uint32_t ww[2] = {w.x, w.y};
        const int bb[2] = {Row::bin_of(x.x), Row::bin_of(x.y)};
#pragma unroll
        for (int h = 0; h < 2; h++)
          if (ww[h] != 0u) {
            const u64 v = widen(ww[h]);
            atomicAdd(&sh.lo[bb[h]], (uint32_t)v & 0xFFFFu);
            atomicAdd(&sh.hi[bb[h]], (uint32_t)(v >> 16));
          }
      }
    }
    __syncthreads();
    for (int b = tid; b < SM_BINS; b += SR_THREADS) {
      const u64 v = ((u64)sh.hi[b] << 16) + sh.lo[b];
      if (v != 0) atomicAdd(&s.mass[b], v);
    }
  } else if (kind == ROW_PLAIN) {
    Sum sum;
#pragma unroll 2
    for (int g = 0; g < G; g++) {
      const Quad q = load_quad(lrow, aligned, v0 + g * SR_GROUP, a.V, lane);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint2 w = row.weight2(make_float2(q.l[e], q.l[e + 1]));
        sum.add(w.x, q.l[e] > -INFINITY && w.x >= row.min_w);
        sum.add(w.y, q.l[e + 1] > -INFINITY && w.y >= row.min_w);
      }
    }
    sum.over_warp();
    if (lane == 0 && v0 < a.V) {
      s.range_w[v0 / SR_RANGE] = sum.w;
      s.range_c[v0 / SR_RANGE] = sum.c;
    }
  }
}

// ---------------------------------------------------------------------------
// the decisions of a row, SM_THREADS threads
// ---------------------------------------------------------------------------
struct RowSmem : ListSmem {
  u64 keys[SR_LIST];
  uint32_t ws[SR_LIST];
  u64 range_w[SR_MAX_RANGES];
  uint32_t range_c[SR_MAX_RANGES];
  int range;
  u64 left;
};

__device__ __forceinline__ void make_hard(const Spaces& sp, RowState* st, int r) {
  if (threadIdx.x == 0) {
    st->kind = ROW_HARD;
    sp.hard[1 + atomicAdd(sp.hard, 1)] = r;
  }
}

// The draw from the masses over SR_RANGE ids in sh.range_w: the range that
// holds the threshold, then its tokens one by one.  Writes token and count.
__device__ void draw_from_ranges(const SampleArgs& a, RowSmem& sh, const Row& row, int ranges, int r) {
  constexpr int PER = SR_MAX_RANGES / SM_THREADS;
  const int tid = threadIdx.x;
  u64 w[PER], mine = 0, all;
  uint32_t cnt = 0;
#pragma unroll
  for (int e = 0; e < PER; e++) {
    const int i = tid * PER + e;
    w[e] = i < ranges ? sh.range_w[i] : 0;
    cnt += i < ranges ? sh.range_c[i] : 0u;
    mine += w[e];
  }
  u64 counted;
  block_prefix(cnt, sh, &counted);
  u64 run = block_prefix(mine, sh, &all) - mine;
  const u64 t = (u64)scaled_threshold(a.u[r], all) + 1;
  if (tid == 0) {  // (always found below; in bounds all the same where a row is written meanwhile)
    sh.range = 0;
    sh.left = 0;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < PER; e++) {
    if (run < t && t <= run + w[e]) {
      sh.range = tid * PER + e;
      sh.left = t - run;
    }
    run += w[e];
  }
  __syncthreads();
  const float* lrow = a.logits + (int64_t)r * a.ld;
  const int id = sh.range * SR_RANGE + 2 * tid;
  static_assert(SR_RANGE == 2 * SM_THREADS, "two tokens a thread");
  const float2 l = make_float2(id < a.V ? lrow[id] : -INFINITY, id + 1 < a.V ? lrow[id + 1] : -INFINITY);
  const uint2 v = row.weight2(l);
  const u64 x = row.inside(l.x, id) && v.x >= row.min_w ? widen(v.x) : 0;
  const u64 y = row.inside(l.y, id + 1) && v.y >= row.min_w ? widen(v.y) : 0;
  const u64 upto = block_prefix(x + y, sh, &all), from = upto - x - y;
  if (from < sh.left && sh.left <= upto) {
    a.token[r] = from + x >= sh.left ? id : id + 1;
    if (a.n_kept != nullptr) a.n_kept[r] = (int)counted;
  }
}

__global__ void __launch_bounds__(SM_THREADS)
sr_cut_kernel(const SampleArgs a, const Spaces sp) {
  extern __shared__ __align__(16) unsigned char dyn[];
  RowSmem& sh = *reinterpret_cast<RowSmem*>(dyn);
  grid_dep_launch();
  const int r = blockIdx.x, tid = threadIdx.x;
  const RowSpace s = sp.row(r);
  grid_dep_wait();
  RowState* st = s.state;
  const int kind = st->kind;
  Row row = st->row;
  if (kind == ROW_PLAIN) {
    for (int i = tid; i < sp.ranges; i += SM_THREADS) {
      sh.range_w[i] = __ldcg(s.range_w + i);
      sh.range_c[i] = __ldcg(s.range_c + i);
    }
    __syncthreads();
    draw_from_ranges(a, sh, row, sp.ranges, r);
  } else if (kind == ROW_TOP_P) {
    constexpr int PER = SM_BINS / SM_THREADS;
    u64 w[PER], mine = 0, S;
#pragma unroll
    for (int e = 0; e < PER; e++) {
      w[e] = __ldcg(s.mass + tid * PER + e);
      mine += w[e];
    }
    u64 run = block_prefix(mine, sh, &S) - mine;
    const u64 need = mass_needed(st->P, S);
#pragma unroll
    for (int e = 0; e < PER; e++) {
      if (run < need && need <= run + w[e]) {
        st->bin = tid * PER + e;
        st->left = need - run;
      }
      run += w[e];
    }
  } else if (kind == ROW_TOP_K) {
    const uint32_t m = st->listed;
    if (m > SR_LIST) {
      make_hard(sp, st, r);
      return;
    }
    for (int i = tid; i < (int)m; i += SM_THREADS) {
      sh.keys[i] = __ldcg(s.key + i);
      sh.ws[i] = __ldcg(s.w + i);
    }
    __syncthreads();
    // the keys agree above the first bit in which the bound and the largest differ
    const uint32_t hi = max_key(st->top), lo = max_key(st->bound);
    const int open = 32 - __clz(hi ^ lo);
    const u64 prefix = open < 32 ? hi >> open : 0u;
    const bool by_p = st->P < (1ull << 32);
    Cut c = cut_list(sh, sh.keys, sh.ws, (int)m, true, by_p, (u64)st->k, 20 + open, prefix);
    if (by_p) c = cut_list(sh, sh.keys, sh.ws, (int)m, false, true, mass_needed(st->P, c.mass), 20 + open, prefix);
    row.set_cut(c.key);
    // the draw: in the order of ids, among the tokens that stay
    u64 mine = 0, S, counted;
    uint32_t cnt = 0;
    for (int i = tid; i < (int)m; i += SM_THREADS) {
      const bool in = sh.keys[i] >= c.key && sh.ws[i] >= row.min_w;
      if (!in) sh.ws[i] = 0u;
      sh.keys[i] &= 0xFFFFFu;  // the lower ids first
      mine += widen(sh.ws[i]);
      cnt += in;
    }
    block_prefix(cnt, sh, &counted);
    block_prefix(mine, sh, &S);
    const u64 t = (u64)scaled_threshold(a.u[r], S) + 1;
    const Cut d = cut_list(sh, sh.keys, sh.ws, (int)m, false, true, t, 20, 0);
    if (tid == 0) {
      a.token[r] = 0xFFFFF - (int)d.key;
      if (a.n_kept != nullptr) a.n_kept[r] = (int)counted;
      st->row = row;
    }
  }
}

// ---------------------------------------------------------------------------
// step and draw of the top-p rows
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(SR_THREADS)
sr_step_kernel(const SampleArgs a, const Spaces sp, int segs) {
  __shared__ OwnList own;
  grid_dep_launch();
  const int r = blockIdx.x / segs, seg = blockIdx.x % segs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RowSpace s = sp.row(r);
  const float* lrow = a.logits + (int64_t)r * a.ld;
  const bool aligned = (reinterpret_cast<uintptr_t>(lrow) & 15u) == 0;
  const int v0 = seg * SR_SEG + warp * SR_RANGE;
  if (tid == 0) own.n = 0;
  __syncthreads();
  grid_dep_wait();
  if (s.state->kind != ROW_TOP_P) return;
  const Row row = s.state->row;
  const int bin = s.state->bin;
  Sum sum;
#pragma unroll 2
  for (int g = 0; g < SR_RANGE / SR_GROUP; g++) {
    const Quad q = load_quad(lrow, aligned, v0 + g * SR_GROUP, a.V, lane);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float2 x = row.x2(make_float2(q.l[e], q.l[e + 1]));
      const int b0 = Row::bin_of(x.x), b1 = Row::bin_of(x.y);
      if (b0 < bin || b1 < bin) {
        const uint2 w = Row::w2(x);
        sum.add(w.x, b0 < bin && w.x >= row.min_w);
        sum.add(w.y, b1 < bin && w.y >= row.min_w);
      }
      if (b0 == bin && q.l[e] > -INFINITY) own_add(own, q.l[e], q.id[e]);
      if (b1 == bin && q.l[e + 1] > -INFINITY) own_add(own, q.l[e + 1], q.id[e + 1]);
    }
  }
  sum.over_warp();
  if (lane == 0 && v0 < a.V) {
    s.range_w[v0 / SR_RANGE] = sum.w;
    s.range_c[v0 / SR_RANGE] = sum.c;
  }
  own_flush(own, s, row);
}

__global__ void __launch_bounds__(SM_THREADS)
sr_draw_kernel(const SampleArgs a, const Spaces sp) {
  extern __shared__ __align__(16) unsigned char dyn[];
  RowSmem& sh = *reinterpret_cast<RowSmem*>(dyn);
  grid_dep_launch();
  const int r = blockIdx.x, tid = threadIdx.x;
  const RowSpace s = sp.row(r);
  grid_dep_wait();
  RowState* st = s.state;
  if (st->kind != ROW_TOP_P) return;
  const uint32_t m = st->listed;
  if (m > SR_LIST) {
    make_hard(sp, st, r);
    return;
  }
  for (int i = tid; i < sp.ranges; i += SM_THREADS) {
    sh.range_w[i] = __ldcg(s.range_w + i);
    sh.range_c[i] = __ldcg(s.range_c + i);
  }
  for (int i = tid; i < (int)m; i += SM_THREADS) {
    sh.keys[i] = __ldcg(s.key + i);
    sh.ws[i] = __ldcg(s.w + i);
  }
  __syncthreads();
  const Cut c = cut_list(sh, sh.keys, sh.ws, (int)m, false, true, st->left, 52, 0);
  Row row = st->row;
  row.set_cut(c.key);
  for (int i = tid; i < (int)m; i += SM_THREADS)
    if (sh.keys[i] >= c.key && sh.ws[i] >= row.min_w) {  // of the step, what stays
      const int range = (0xFFFFF - (int)(sh.keys[i] & 0xFFFFFu)) / SR_RANGE;
      atomicAdd(&sh.range_w[range], widen(sh.ws[i]));
      atomicAdd(&sh.range_c[range], 1u);
    }
  __syncthreads();
  if (tid == 0) st->row = row;
  draw_from_ranges(a, sh, row, sp.ranges, r);
}

// ---------------------------------------------------------------------------
// filter
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(SR_THREADS)
sr_filter_kernel(const SampleArgs a, const Spaces sp, int segs) {
  const int r = blockIdx.x / segs, seg = blockIdx.x % segs;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RowState* st = sp.row(r).state;
  const float* lrow = a.logits + (int64_t)r * a.ld;
  float* frow = a.filtered + (int64_t)r * a.ldf;
  const bool aligned =
      ((reinterpret_cast<uintptr_t>(lrow) | reinterpret_cast<uintptr_t>(frow)) & 15u) == 0;
  const int v0 = seg * SR_SEG + warp * SR_RANGE;
  grid_dep_wait();
  const int kind = st->kind;
  if (kind == ROW_HARD) return;  // written by its cluster
  const Row row = st->row;
#pragma unroll 4
  for (int g = 0; g < SR_RANGE / SR_GROUP; g++) {
    const int g0 = v0 + g * SR_GROUP;
    const Quad q = load_quad(lrow, aligned, g0, a.V, lane);
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      bool in = row.inside(q.l[e], q.id[e]);
      if (in && row.min_w != 0u) in = row.weight(q.l[e]) >= row.min_w;
      o[e] = kind == ROW_BAD ? __int_as_float(0x7FFFFFFF) : in ? q.l[e] : SPEC_FILTERED;
    }
    if (aligned && g0 + SR_GROUP <= a.V) {
      __stcs(reinterpret_cast<float4*>(frow + g0) + lane, make_float4(o[0], o[1], o[2], o[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (q.id[e] < a.V) frow[q.id[e]] = o[e];
    }
  }
}

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), size_t grid, int threads, size_t smem, cudaStream_t st, bool dependent,
                   A... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = dependent && programmatic_launch() ? 1 : 0;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

size_t sample_rows_bytes(int R, int V) {
  const Spaces s = spaces(nullptr, R, V);
  return (size_t)(s.base - (char*)nullptr) + s.stride * R;
}

void sample_rows_init_attrs() {
  int dev = 0, optin = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  cudaFuncSetAttribute(sr_cut_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
  cudaFuncSetAttribute(sr_draw_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
}

int sample_rows_launch(SampleArgs a, void* workspace, cudaStream_t st) {
  const Spaces sp = spaces(workspace, a.R, a.V);
  const int segs = (a.V + SR_SEG - 1) / SR_SEG;
  const size_t grid = (size_t)a.R * segs;
  if (grid > INT32_MAX) return fail(SPEC_E_SHAPE, "sample: R * V too large");
  cudaError_t e = launch(sr_maxima_kernel, grid, SR_THREADS, 0, st, false, a, sp, segs);
  if (e == cudaSuccess)
    e = launch(sr_bound_kernel, a.R, SR_THREADS, sizeof(uint32_t) * sp.groups, st, true, a, sp);
  if (e == cudaSuccess) e = launch(sr_pass_kernel, grid, SR_THREADS, 0, st, true, a, sp, segs);
  if (e == cudaSuccess) e = launch(sr_cut_kernel, a.R, SM_THREADS, sizeof(RowSmem), st, true, a, sp);
  if (e == cudaSuccess && a.top_p != nullptr) {
    e = launch(sr_step_kernel, grid, SR_THREADS, 0, st, true, a, sp, segs);
    if (e == cudaSuccess) e = launch(sr_draw_kernel, a.R, SM_THREADS, sizeof(RowSmem), st, true, a, sp);
  }
  if (e == cudaSuccess && a.filtered != nullptr)
    e = launch(sr_filter_kernel, grid, SR_THREADS, 0, st, true, a, sp, segs);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("sample: ") + cudaGetErrorString(e));
  // (an ordinary launch: behind everything in front of it)
  a.rows = sp.hard + 1;
  a.n_rows = sp.hard;
  return sample_clusters_launch(a, std::min(a.R, SR_HARD_CLUSTERS), st);
}
