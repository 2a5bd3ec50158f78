// sample_rows.cu -- filtered sampling of many long rows: passes over all of
// them (the same rules and integer sums as sample.cu, which keeps a row in the
// shared memory of a cluster and is bound by its barriers, not by the memory,
// once rows are many).
//
// A row is one of three kinds, by its settings: top-k (with or without the
// other filters), top-p alone, or neither.  Streaming passes have a CTA per
// 8192 or 16384 logits of a row, a warp per 1024 of them at a time; between
// them a CTA per row decides.
//   maxima   stream: the largest logit of every 128, and of groups of 16 .. 128
//   bound    row: the largest, the settings, and for a top-k a bound that at
//            least k of these groups reach
//   pass     stream: top-k rows collect the tokens at the bound (only blocks
//            of 128 that reach it are read); top-p rows add their masses up
//            over steps of z; the others over 1024 ids
//   cut      row, top-p rows: the step that holds the cut
//   step     stream, top-p rows: the masses above that step over 1024 ids,
//            its tokens collected
//   draw     row: the cut among the collected tokens, and the draw from these
//            (top-k), from the masses over ids (no filter) or both (top-p)
//   filter   stream, where filtered logits are wanted: blocks below the cut
//            are written without being read
// A row that collects too many tokens goes to the clusters of sample.cu as a
// whole.  Each kernel is a programmatic dependent of the one in front of it,
// and every other stream runs from the last row to the first, to find in L2
// what the one before read last.
//
// Measured, 192 rows of 248320 logits (191 MB, 28 us at the copy bandwidth):
// without filters 90 us, with a top-k 79, with all filters 82, with a top-p
// alone 174, rows of mixed settings 117 (in clusters 380); 48 to 77 more where
// filtered logits are written (another 191 MB).  maxima 30 us: the memory.
// pass 51 (no filter: 17 instructions a weight and the sums), 30 (top-k: the
// blocks that reach the bound), 63 (top-p: two 32-bit additions in shared
// memory a logit).  step 61 (top-p).  filter 38 to 64.  bound 5 to 9, cut 5,
// draw 6 to 14: a CTA a row, latency.
#include <algorithm>

#include "sample.cuh"

namespace {

constexpr int SR_BLOCK = 128;  // logits of a warp's load
// Groups whose largest bound a top-k: 1, 2, 4 or 8 of a block, as many as make
// no more than SR_MAX_GROUPS.
constexpr int SR_MAX_GROUPS = 8192;
constexpr int SR_RANGE = 1024;  // logits of a warp, and ids whose mass is kept
constexpr int SR_WARPS = 8;
constexpr int SR_THREADS = 32 * SR_WARPS;
constexpr int SR_SEG = SR_RANGE * SR_WARPS;
constexpr int SR_LIST = 4096;  // tokens that are collected of a row
constexpr int SR_MAX_RANGES = 1024;
constexpr int SR_BOUND_BITS = 9, SR_BOUND_BINS = 1 << SR_BOUND_BITS;
static_assert(SR_BOUND_BINS == SM_THREADS, "a bin a thread");
// Clusters for the rows that do not fit the list, in turns.  Flat rows are such:
// top-p rows of 248320 logits whose deviation is below about 0.4 T have more
// than SR_LIST tokens in the step that holds their cut.  A cluster's refinement
// adds to few bins then, so that a row takes about 180 us of it: 192 of them 2.4
// ms (deviation 0.3 T), 0.23 at 0.5 T and 0.17 at 2 T.
constexpr int SR_HARD_CLUSTERS = 16;

enum RowKind : int { ROW_BAD, ROW_PLAIN, ROW_TOP_K, ROW_TOP_P, ROW_HARD };

struct RowState {
  Row row;  // (the cut in it where there is one: from the kernel that finds it on)
  float top;
  float bound;   // top-k: tokens from here on are collected; top-p: from here on up to
  float summed;  // here, and from here on their masses are summed up
  int kind, k;
  u64 P;
  u64 left;  // top-p: the mass to reach inside the step
  uint32_t listed;
};

// One row's workspace.
struct RowSpace {
  RowState* state;
  uint32_t* block;  // order keys of the largest of SR_BLOCK logits
  uint32_t* group;  // and of each group (the same where a block is one)
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
  int blocks, groups, ranges;
  int per;  // groups of a block
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
    s.block = reinterpret_cast<uint32_t*>(p);
    s.group = per == 1 ? s.block : s.block + blocks;
    return s;
  }
};

Spaces spaces(void* workspace, int R, int V) {
  Spaces s;
  s.blocks = (V + SR_BLOCK - 1) / SR_BLOCK;
  s.per = 8;
  while (s.blocks * s.per > SR_MAX_GROUPS) s.per /= 2;
  s.groups = s.blocks * s.per;
  s.ranges = (V + SR_RANGE - 1) / SR_RANGE;
  s.stride = Spaces::up(sizeof(RowState)) + Spaces::up(sizeof(u64) * SM_BINS) + Spaces::up(sizeof(u64) * SR_LIST) +
             Spaces::up(sizeof(uint32_t) * SR_LIST) + Spaces::up(sizeof(u64) * s.ranges) +
             Spaces::up(sizeof(uint32_t) * s.ranges) + Spaces::up(sizeof(uint32_t) * (s.blocks + s.groups));
  s.hard = reinterpret_cast<int32_t*>(workspace);
  s.base = reinterpret_cast<char*>(workspace) + Spaces::up(sizeof(int32_t) * ((size_t)R + 1));
  return s;
}

// A lane's four logits of each of the warp's blocks, from id v0 on: ids
// 4 lane .. of a block (16-byte loads) where the rows are aligned and the block
// is whole, else lane + 32 e.
constexpr int SR_BLOCKS = SR_RANGE / SR_BLOCK;  // of a warp
template <int N>
struct Logits {
  float4 l[N];
  int v0, V, lane;
  bool aligned;
  __device__ __forceinline__ Logits(const void* row, int v0_, int V_)
      : v0(v0_), V(V_), lane(threadIdx.x & 31), aligned((reinterpret_cast<uintptr_t>(row) & 15u) == 0) {}
  __device__ __forceinline__ bool whole(int g) const { return aligned && v0 + (g + 1) * SR_BLOCK <= V; }
  __device__ __forceinline__ int id(int g, int e) const {
    return v0 + g * SR_BLOCK + (whole(g) ? 4 * lane + e : lane + 32 * e);
  }
  // the blocks of `which` (a bit each)
  __device__ __forceinline__ void load(const float* row, uint32_t which) {
    if (which == (1u << N) - 1u && whole(N - 1)) {
#pragma unroll
      for (int g = 0; g < N; g++) l[g] = reinterpret_cast<const float4*>(row + v0 + g * SR_BLOCK)[lane];
      return;
    }
#pragma unroll
    for (int g = 0; g < N; g++) {
      l[g] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (which >> g & 1u) {
        if (whole(g)) {
          l[g] = reinterpret_cast<const float4*>(row + v0 + g * SR_BLOCK)[lane];
        } else {
          const int at = v0 + g * SR_BLOCK + lane;
          if (at < V) l[g].x = row[at];
          if (at + 32 < V) l[g].y = row[at + 32];
          if (at + 64 < V) l[g].z = row[at + 64];
          if (at + 96 < V) l[g].w = row[at + 96];
        }
      }
    }
  }
};
// The blocks of the warp's turns whose largest logit is at least
// `least`: eight bits a turn.
constexpr int SR_TURNS = 2;  // at most: segments of a CTA
__device__ __forceinline__ uint32_t blocks_from(const Spaces& sp, const RowSpace& s, int v0, float least) {
  const int lane = threadIdx.x & 31, at = (v0 + (lane >> 3) * SR_SEG) / SR_BLOCK + (lane & 7);
  const uint32_t key = at < sp.blocks ? __ldcg(s.block + at) : 0u;
  return __ballot_sync(0xffffffffu, key >= max_key(least));
}

// The warp's turns by halves: each(half, its blocks of `blocks`), and after each
// turn done(its first id).  Half the registers, so that five or six CTAs are
// resident: mixed rows with filtered logits 191 us with whole turns and four,
// 177 by halves; 215 with a half's loads in front of the other's work.
constexpr int SR_HALF = SR_BLOCKS / 2;
typedef Logits<SR_HALF> Half;
template <class Each, class Done>
__device__ __forceinline__ void by_halves(const float* row, Half& a, int turns, uint32_t blocks, Each&& each,
                                          Done&& done) {
  constexpr uint32_t ALL = (1u << SR_HALF) - 1u;
  for (int turn = 0; turn < turns; turn++, a.v0 += SR_SEG - SR_RANGE) {
#pragma unroll 1
    for (int half = 0; half < 2; half++, a.v0 += SR_RANGE / 2, blocks >>= SR_HALF) {
      a.load(row, blocks & ALL);
      each(a, blocks & ALL);
    }
    done(a.v0 - SR_RANGE);
  }
}

// ---------------------------------------------------------------------------
// maxima
// ---------------------------------------------------------------------------
constexpr uint32_t NAN_KEY = 0xFFFFFFFFu;  // above every key
__device__ __forceinline__ float nan_max(float x, float y) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(y));
  return x;
}
__global__ void __launch_bounds__(SR_THREADS)
sr_maxima_kernel(const SampleArgs a, const Spaces sp, int segs) {
  grid_dep_begin();  // (what comes next reads the settings in front of its wait)
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
  const int v0 = seg * SR_SEG + warp * SR_RANGE;
  Logits<SR_BLOCKS> q(row, v0, a.V);
  q.load(row, (1u << SR_BLOCKS) - 1u);
  uint32_t mx[SR_BLOCKS];  // order keys, NAN_KEY for a NaN (of which the bits of a sum say nothing)
#pragma unroll
  for (int g = 0; g < SR_BLOCKS; g++) {
    float m = nan_max(nan_max(q.l[g].x, q.l[g].y), nan_max(q.l[g].z, q.l[g].w));
    m = nan_max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = nan_max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    mx[g] = m != m ? NAN_KEY : max_key(m);
  }
  static_assert(SR_BLOCKS == 8, "two blocks a lane of four");
  const int b0 = v0 / SR_BLOCK;
  if (sp.per > 1) {
    int each = 4;  // lanes of a group
    for (; each * sp.per < 32; each *= 2)
#pragma unroll
      for (int g = 0; g < SR_BLOCKS; g++) mx[g] = max(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], each));
    // the group's lanes 0 .. 3: blocks i and i + 4
    uint32_t lo = mx[0], hi = mx[4];
#pragma unroll
    for (int i = 1; i < 4; i++) {
      lo = (lane & 3) == i ? mx[i] : lo;
      hi = (lane & 3) == i ? mx[4 + i] : hi;
    }
    const int at = b0 + (lane & 3), group = lane / each;
    if (lane % each < 4) {
      if (at < sp.blocks) s.group[at * sp.per + group] = lo;
      if (at + 4 < sp.blocks) s.group[(at + 4) * sp.per + group] = hi;
    }
  }
  uint32_t mine = 0u;
#pragma unroll
  for (int g = 0; g < SR_BLOCKS; g++) {
    const uint32_t all = __reduce_max_sync(0xffffffffu, mx[g]);
    mine = lane == g ? all : mine;
  }
  if (lane < SR_BLOCKS && b0 + lane < sp.blocks) s.block[b0 + lane] = mine;
}

// ---------------------------------------------------------------------------
// bound
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(SM_THREADS)
sr_bound_kernel(const SampleArgs a, const Spaces sp) {
  __shared__ uint32_t s_top[SM_WARPS], s_low[SM_WARPS], s_cnt[SR_BOUND_BINS], s_from;
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
  // the groups' keys, of finite logits (0 for the others), and their range
  constexpr uint32_t NONE = 0x007FFFFFu;  // key of -infinity
  uint32_t key[SR_MAX_GROUPS / SM_THREADS], top = 0, least = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < SR_MAX_GROUPS / SM_THREADS; i++) {
    const int g = i * SM_THREADS + tid;
    key[i] = g < sp.groups ? __ldcg(s.group + g) : 0u;
    if (key[i] <= NONE) key[i] = 0u;
    top = max(top, key[i]);
    least = min(least, key[i] - 1u);  // (0 is the largest)
  }
  top = __reduce_max_sync(0xffffffffu, top);
  least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 0) {
    s_top[warp] = top;
    s_low[warp] = least;
  }
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, s_top[lane % SM_WARPS]);
  least = __reduce_min_sync(0xffffffffu, s_low[lane % SM_WARPS]) + 1u;
  const bool finite = top > NONE && top < 0xFF800000u;  // below +infinity and NaN
  st.top = finite ? key_value(top) : 0.0f;
  row.zmax = row_zmax(max_key(st.top), row.T);
  row.plain |= Row::far(row.zmax);
  bad |= !finite || !(fabsf(row.zmax) < INFINITY);
  const bool by_k = st.k > 0 && st.k < a.V;
  st.bound = -INFINITY;
  st.kind = bad ? ROW_BAD : by_k ? ROW_HARD : st.P < (1ull << 32) ? ROW_TOP_P : ROW_PLAIN;
  // how many tokens would be collected, were logits independent: groups of n
  // are below the bound with the chance 1 - k / groups
  const float n = (float)(SR_BLOCK / sp.per), part = (float)st.k / (float)sp.groups;
  if (!bad && by_k && part < 1.0f && n * sp.groups * (1.0f - powf(1.0f - part, 1.0f / n)) < 0.9f * SR_LIST) {
    // the k-th largest of the keys, nine bits a step from the first that
    // differs; after two steps what is left of the bits is taken as 0
    const int open = 32 - __clz(top ^ least);
    int down = open;
    uint32_t from = open < 32 ? top >> open : 0u, left = (uint32_t)st.k;
    bool enough = true;
    for (int step = 0; step < 2 && down > 0 && enough; step++) {
      const int above = down;
      down = max(0, down - SR_BOUND_BITS);
      const uint32_t mask = (1u << (above - down)) - 1u;
      s_cnt[tid] = 0u;
      if (tid == 0) s_from = 0xFFFFFFFFu;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < SR_MAX_GROUPS / SM_THREADS; i++)
        if (key[i] != 0u && (above == 32 || key[i] >> above == from))
          atomicAdd(&s_cnt[SR_BOUND_BINS - 1 - (key[i] >> down & mask)], 1u);
      __syncthreads();
      const uint32_t c = s_cnt[tid];
      uint32_t run = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += y;
      }
      if (lane == 31) s_top[warp] = run;
      __syncthreads();
      run += __reduce_add_sync(0xffffffffu, lane < warp ? s_top[lane] : 0u);
      if (run - c < left && left <= run) {
        s_from = from << (above - down) | (uint32_t)(SR_BOUND_BINS - 1 - tid);
        s_low[0] = left - (run - c);
      }
      __syncthreads();
      enough = s_from != 0xFFFFFFFFu;  // at least k groups have a finite logit
      from = s_from;
      left = s_low[0];
      __syncthreads();
    }
    if (open == 0) enough = false;  // (all alike: more than a list of them)
    if (enough) {
      st.bound = key_value(from << down);
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
  u64 key[SR_LIST];
  uint32_t n, at;
};
__device__ __forceinline__ void own_add(OwnList& o, float l, int id) {
  const uint32_t at = atomicAdd(&o.n, 1u);
  if (at < SR_LIST) o.key[at] = Row::composite(max_key(l), id);
}
__device__ __forceinline__ void own_flush(OwnList& o, const RowSpace& s, const Row& row) {
  __syncthreads();
  const uint32_t n = o.n;
  if (threadIdx.x == 0 && n > 0) o.at = atomicAdd(&s.state->listed, min(n, SR_LIST + 1u));
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < min(n, (uint32_t)SR_LIST); c += SR_THREADS)
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
    if (in) {
      w += x;
      w += x == 0xFFFFFFFFu;
      c++;
    }
  }
  __device__ __forceinline__ void store(const RowSpace& s, int v0, int V) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0 && v0 < V) {
      s.range_w[v0 / SR_RANGE] = w;
      s.range_c[v0 / SR_RANGE] = c;
    }
    w = 0;
    c = 0;
  }
};

__global__ void __launch_bounds__(SR_THREADS, 5)
sr_pass_kernel(const SampleArgs a, const Spaces sp, int segs, int turns) {
  __shared__ union {
    struct {
      uint32_t lo[SM_BINS], hi[SM_BINS];
    };
    OwnList own;
  } sh;
  grid_dep_launch();
  const int at = (int)(gridDim.x - 1 - blockIdx.x), r = at / segs, seg = at % segs;
  const int tid = threadIdx.x, warp = tid >> 5;
  const RowSpace s = sp.row(r);
  const float* lrow = a.logits + (int64_t)r * a.ld;
  Half q(lrow, (seg * turns * SR_WARPS + warp) * SR_RANGE, a.V);
  grid_dep_wait();
  const int kind = s.state->kind;
  const Row row = s.state->row;
  if (kind == ROW_TOP_K) {
    const float bound = s.state->bound;
    if (tid == 0) sh.own.n = 0;
    __syncthreads();
    by_halves(lrow, q, turns, blocks_from(sp, s, q.v0, bound),
              [&](const Half& h, uint32_t which) {
                if (which == 0u) return;
#pragma unroll
                for (int g = 0; g < SR_HALF; g++) {
                  const float l[4] = {h.l[g].x, h.l[g].y, h.l[g].z, h.l[g].w};
#pragma unroll
                  for (int e = 0; e < 4; e++)
                    if (l[e] >= bound) own_add(sh.own, l[e], h.id(g, e));
                }
              },
              [](int) {});
    own_flush(sh.own, s, row);
  } else if (kind == ROW_TOP_P) {
    for (int b = tid; b < SM_BINS; b += SR_THREADS) sh.lo[b] = sh.hi[b] = 0;
    __syncthreads();
    by_halves(lrow, q, turns, ~0u,
              [&](const Half& h, uint32_t) {
#pragma unroll
                for (int g = 0; g < SR_HALF; g++) {
                  const float2 l[2] = {make_float2(h.l[g].x, h.l[g].y), make_float2(h.l[g].z, h.l[g].w)};
#pragma unroll
                  for (int e = 0; e < 2; e++) {
                    const float2 x = row.x2(l[e]);
                    const uint2 w = Row::w2(x);
                    const uint32_t ww[2] = {w.x, w.y};
                    const int bb[2] = {Row::bin_of(x.x), Row::bin_of(x.y)};
#pragma unroll
                    for (int k = 0; k < 2; k++)
                      if (ww[k] != 0u) {
                        const u64 v = widen(ww[k]);
                        atomicAdd(&sh.lo[bb[k]], (uint32_t)v & 0xFFFFu);
                        atomicAdd(&sh.hi[bb[k]], (uint32_t)(v >> 16));
                      }
                  }
                }
              },
              [](int) {});
    __syncthreads();
    for (int b = tid; b < SM_BINS; b += SR_THREADS) {
      const u64 v = ((u64)sh.hi[b] << 16) + sh.lo[b];
      if (v != 0) atomicAdd(&s.mass[b], v);
    }
  } else if (kind == ROW_PLAIN) {
    Sum sum;
    by_halves(lrow, q, turns, ~0u,
              [&](const Half& h, uint32_t) {
#pragma unroll
                for (int g = 0; g < SR_HALF; g++) {
                  const float2 l[2] = {make_float2(h.l[g].x, h.l[g].y), make_float2(h.l[g].z, h.l[g].w)};
#pragma unroll
                  for (int e = 0; e < 2; e++) {
                    const uint2 w = row.weight2(l[e]);
                    sum.add(w.x, l[e].x > -INFINITY && w.x >= row.min_w);
                    sum.add(w.y, l[e].y > -INFINITY && w.y >= row.min_w);
                  }
                }
              },
              [&](int v0) { sum.store(s, v0, a.V); });
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

// The least float whose step of z is at most `target`, by a warp: five bits a
// turn of the largest order key with a later step (a step never rises with the
// logit, as each rounding keeps the order).
__device__ __forceinline__ float first_of_step(const Row& row, float top, int target) {
  const int lane = threadIdx.x & 31;
  const uint32_t last = max_key(top);
  uint32_t base = 0u;
  for (int shift = 27;; shift = max(0, shift - 5)) {
    const uint32_t key = base + ((uint32_t)lane << shift);
    bool later = key < 0x00800000u;  // -infinity and what is below it
    if (!later && key <= last) later = row.bin(key_value(key)) > target;
    // (in the last turn lanes 4 .. 31 lie past a key that is known not to be later)
    const uint32_t yes = __ballot_sync(0xffffffffu, later && key >= base);
    base += (uint32_t)(31 - __clz(yes)) << shift;
    if (shift == 0) break;
  }
  return key_value(base + 1u);
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

// A top-p row's step that holds its cut.
__global__ void __launch_bounds__(SM_THREADS)
sr_cut_kernel(const SampleArgs a, const Spaces sp) {
  __shared__ ListSmem sh;
  __shared__ int s_step;
  grid_dep_launch();
  const int tid = threadIdx.x;
  const RowSpace s = sp.row(blockIdx.x);
  grid_dep_wait();
  RowState* st = s.state;
  if (st->kind != ROW_TOP_P) return;
  const Row row = st->row;
  constexpr int PER = SM_BINS / SM_THREADS;
  u64 w[PER], mine = 0, S;
#pragma unroll
  for (int e = 0; e < PER; e++) {
    w[e] = __ldcg(s.mass + tid * PER + e);
    mine += w[e];
  }
  u64 run = block_prefix(mine, sh, &S) - mine;
  const u64 need = mass_needed(st->P, S);
  if (tid == 0) s_step = SM_BINS - 1;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < PER; e++) {
    if (run < need && need <= run + w[e]) {
      s_step = tid * PER + e;
      st->left = need - run;
    }
    run += w[e];
  }
  __syncthreads();
  if (tid < 64) {
    const float first = first_of_step(row, st->top, s_step - (tid >> 5));
    if (tid == 0) st->bound = first;
    if (tid == 32) st->summed = s_step == 0 ? INFINITY : first;
  }
}

// The cut of a top-k row among its collected tokens, and the draw from them.
__device__ void cut_and_draw(const SampleArgs& a, const Spaces& sp, const RowSpace& s, RowSmem& sh, int r) {
  const int tid = threadIdx.x;
  RowState* st = s.state;
  Row row = st->row;
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

// ---------------------------------------------------------------------------
// the step of the top-p rows, and the draw
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(SR_THREADS, 5)
sr_step_kernel(const SampleArgs a, const Spaces sp, int segs, int turns) {
  __shared__ OwnList own;
  grid_dep_launch();
  const int r = blockIdx.x / segs, seg = blockIdx.x % segs;
  const int tid = threadIdx.x, warp = tid >> 5;
  const RowSpace s = sp.row(r);
  const float* lrow = a.logits + (int64_t)r * a.ld;
  Half q(lrow, (seg * turns * SR_WARPS + warp) * SR_RANGE, a.V);
  if (tid == 0) own.n = 0;
  __syncthreads();
  grid_dep_wait();
  if (s.state->kind != ROW_TOP_P) return;
  const Row row = s.state->row;
  const float bound = s.state->bound, summed = s.state->summed;
  Sum sum;
  by_halves(lrow, q, turns, blocks_from(sp, s, q.v0, bound),
            [&](const Half& h, uint32_t which) {
              if (which == 0u) return;
              // a bit for each of the lane's logits; few of a row are above its
              // cut, so that a lane weighs its own, read again, rather than all
              // in turn
              uint32_t above = 0u, within = 0u;
#pragma unroll
              for (int g = 0; g < SR_HALF; g++) {
                const float l[4] = {h.l[g].x, h.l[g].y, h.l[g].z, h.l[g].w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                  if (l[e] >= summed) above |= 1u << (4 * g + e);
                  if (l[e] >= bound) within |= 1u << (4 * g + e);
                }
              }
              within &= ~above;
              while (above != 0u) {
                const int i = __ffs(above) - 1;
                above &= above - 1u;
                const bool two = above != 0u;
                const int j = two ? __ffs(above) - 1 : i;
                above &= above - 1u;
                const uint2 w = row.weight2(make_float2(lrow[h.id(i >> 2, i & 3)], lrow[h.id(j >> 2, j & 3)]));
                sum.add(w.x, w.x >= row.min_w);
                sum.add(w.y, two && w.y >= row.min_w);
              }
              while (within != 0u) {
                const int i = __ffs(within) - 1;
                within &= within - 1u;
                const int id = h.id(i >> 2, i & 3);
                own_add(own, lrow[id], id);
              }
            },
            [&](int v0) {
              __syncwarp();
              sum.store(s, v0, a.V);
            });
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
  const int kind = st->kind;
  if (kind == ROW_TOP_K) cut_and_draw(a, sp, s, sh, r);
  if (kind != ROW_PLAIN && kind != ROW_TOP_P) return;
  for (int i = tid; i < sp.ranges; i += SM_THREADS) {
    sh.range_w[i] = __ldcg(s.range_w + i);
    sh.range_c[i] = __ldcg(s.range_c + i);
  }
  if (kind == ROW_PLAIN) {
    __syncthreads();
    draw_from_ranges(a, sh, st->row, sp.ranges, r);
    return;
  }
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
__global__ void __launch_bounds__(SR_THREADS, 6)
sr_filter_kernel(const SampleArgs a, const Spaces sp, int segs, int turns) {
  const int at = (int)(gridDim.x - 1 - blockIdx.x), r = at / segs, seg = at % segs;
  const int warp = threadIdx.x >> 5;
  const RowSpace s = sp.row(r);
  const float* lrow = a.logits + (int64_t)r * a.ld;
  float* frow = a.filtered + (int64_t)r * a.ldf;
  Half q(lrow, (seg * turns * SR_WARPS + warp) * SR_RANGE, a.V);
  q.aligned = q.aligned && (reinterpret_cast<uintptr_t>(frow) & 15u) == 0;
  grid_dep_wait();
  const int kind = s.state->kind;
  if (kind == ROW_HARD) return;  // written by its cluster
  const Row row = s.state->row;
  const float out = kind == ROW_BAD ? __int_as_float(0x7FFFFFFF) : SPEC_FILTERED;
  auto put = [&](float l, int id) {
    bool in = row.inside(l, id);
    if (in && row.min_w != 0u) in = row.weight(l) >= row.min_w;
    return in ? l : out;
  };
  by_halves(lrow, q, turns, kind == ROW_BAD ? 0u : blocks_from(sp, s, q.v0, row.least),
            [&](const Half& h, uint32_t which) {
#pragma unroll
              for (int g = 0; g < SR_HALF; g++) {
                float4 l = make_float4(out, out, out, out);
                if (which >> g & 1u)
                  l = make_float4(put(h.l[g].x, h.id(g, 0)), put(h.l[g].y, h.id(g, 1)), put(h.l[g].z, h.id(g, 2)),
                                  put(h.l[g].w, h.id(g, 3)));
                if (h.whole(g)) {
                  reinterpret_cast<float4*>(frow + h.v0 + g * SR_BLOCK)[h.lane] = l;
                } else {
                  const float e[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                  for (int k = 0; k < 4; k++)
                    if (h.id(g, k) < a.V) frow[h.id(g, k)] = e[k];
                }
              }
            },
            [](int) {});
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
  cudaFuncSetAttribute(sr_draw_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
}

int sample_rows_launch(SampleArgs a, void* workspace, cudaStream_t st) {
  const Spaces sp = spaces(workspace, a.R, a.V);
  const int segs = (a.V + SR_SEG - 1) / SR_SEG;
  const size_t grid = (size_t)a.R * segs;
  if (grid > INT32_MAX) return fail(SPEC_E_SHAPE, "sample: R * V too large");
  // two segments a CTA where CTAs are many, eight an SM and more of them (192
  // rows of 248320 logits, a top-k: 86 us with one, 78 with two, 76 with four,
  // which end unevenly, though, where rows are of different kinds)
  const int turns = (int)std::max<size_t>(1, std::min<size_t>(SR_TURNS, grid / (8 * device_sms())));
  const int long_segs = (segs + turns - 1) / turns;
  const size_t long_grid = (size_t)a.R * long_segs;
  cudaError_t e = launch_dependent(sr_maxima_kernel, grid, SR_THREADS, 0, st, a, sp, segs);
  if (e == cudaSuccess)
    e = launch_dependent(sr_bound_kernel, a.R, SM_THREADS, 0, st, a, sp);
  if (e == cudaSuccess) e = launch_dependent(sr_pass_kernel, long_grid, SR_THREADS, 0, st, a, sp, long_segs, turns);
  if (e == cudaSuccess && a.top_p != nullptr) {
    e = launch_dependent(sr_cut_kernel, a.R, SM_THREADS, 0, st, a, sp);
    if (e == cudaSuccess) e = launch_dependent(sr_step_kernel, long_grid, SR_THREADS, 0, st, a, sp, long_segs, turns);
  }
  if (e == cudaSuccess) e = launch_dependent(sr_draw_kernel, a.R, SM_THREADS, sizeof(RowSmem), st, a, sp);
  if (e == cudaSuccess && a.filtered != nullptr)
    e = launch_dependent(sr_filter_kernel, long_grid, SR_THREADS, 0, st, a, sp, long_segs, turns);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("sample: ") + cudaGetErrorString(e));
  a.rows = sp.hard + 1;
  a.n_rows = sp.hard;
  return sample_clusters_launch(a, std::min(a.R, SR_HARD_CLUSTERS), st);
}
