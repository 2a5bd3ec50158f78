// tree_attn.cuh -- what the tree attention kernels share: their arguments, the
// cut of the work over the CTAs, a tree's ancestors.  Internal.
#pragma once

#include <stdint.h>

#include "common.cuh"

struct TreeArgs {
  const __half* k;  // the layer's cache
  const __half* v;
  const int32_t* table;
  const int32_t* len;
  int n_slots, max_pages, n_pages, nkv, page_size, page_shift;  // shift -1: not a power of two
  const int32_t* slots;
  const int32_t* parents;
  const int32_t* n_nodes;
  int n_seq, nt, nq, G, window, sinks;
  float scale_log2;
  const __half* q;
  int64_t q_stride;
  const __half* k_new;
  const __half* v_new;
  int64_t kv_stride;
  __half* out;
  uint32_t g_inv;  // ceil(2^32 / G): m / G = umulhi(m, g_inv) for m G < 2^32 and G > 1
  int rows;        // query rows of a unit (16 to 256, a power of two)
  int tile_shift;  // log2 of the positions of a tile
  float* part_o;    // [N][2][HD / 4][rows][4]: a lane a row, its stores side by side
  float2* part_ml;  // [N][2][rows]
  uint32_t* part_err;  // [N]: 1 if the CTA gave up on a wait
  struct TreePlan* plan;  // [n_seq]
  int32_t* status;
};

// One sequence's part of the cut, for the joining kernel.
struct TreePlan {
  long long before;  // tiles of the sequences in front of it
  long long share;   // tiles of a CTA
  int tiles;         // of each of its units
  int nodes;         // rows of the output that are the call's to write
  int status;
  int pad;
};

namespace {

// ---------------------------------------------------------------------------
// the cut of the work
// ---------------------------------------------------------------------------
// One sequence: its tiles are the sink tiles below the window, the tiles from
// the window's first position to the last, and the tree's own.
struct SeqInfo {
  int slot, len, m;
  int lo;       // first position that some node's window reaches
  int sinks;    // positions of the prefix that stay visible under a window
  int w_tile;   // tile of lo
  int n_sink;   // sink tiles in front of it
  int tiles;
  int units;    // kv heads x row blocks
  int bad;      // status bits of what is checked here
  __device__ __forceinline__ long long work() const { return (long long)units * tiles; }
};

__device__ __forceinline__ SeqInfo seq_info(const TreeArgs& a, int s, int rows, int tile_shift) {
  SeqInfo q;
  q.slot = a.slots[s];
  q.m = a.n_nodes != nullptr ? a.n_nodes[s] : a.nt;
  q.bad = 0;
  q.len = 0;
  if (q.slot < 0 || q.slot >= a.n_slots) {
    q.bad |= SPEC_ST_SLOT;
  } else {
    q.len = a.len[q.slot];
    if (q.len < 0 || q.len > a.max_pages * a.page_size) q.bad |= SPEC_ST_PAGE;
  }
  if (q.m < 0 || q.m > a.nt) q.bad |= SPEC_ST_TREE;
  if (q.bad != 0) q.len = q.m = 0;
  q.lo = a.window > 0 ? max(0, q.len - a.window + 1) : 0;
  q.sinks = a.window > 0 ? min(a.sinks, q.len) : 0;
  const int up = (1 << tile_shift) - 1, end = (q.len + up) >> tile_shift;
  q.w_tile = q.lo < q.len ? q.lo >> tile_shift : end;
  q.n_sink = min((q.sinks + up) >> tile_shift, q.w_tile);
  q.tiles = q.n_sink + (end - q.w_tile) + 1;
  q.units = q.m > 0 ? a.nkv * ((q.m * a.G + rows - 1) / rows) : 0;
  return q;
}

// Exclusive sum over the CTA's threads; *total: the whole.
template <int THREADS>
__device__ __forceinline__ long long block_excl(long long v, long long* s_part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 31) s_part[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; w++) {
    if (w < warp) before += s_part[w];
    all += s_part[w];
  }
  *total = all;
  return before + x - v;
}

// a / b for non-negative values: 64-bit division is a long subroutine, and
// all but enormous calls have less than 2^32 tiles.
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  if ((((unsigned long long)a | (unsigned long long)b) >> 32) == 0)
    return (long long)((unsigned)a / (unsigned)b);
  return a / b;
}

// Tiles of a CTA: CTA b takes [b * share, (b + 1) * share) of the total.
__device__ __forceinline__ long long share_of(long long total, int n) {
  return div_ll(total + n - 1, n);
}

__device__ __forceinline__ int node_of(const TreeArgs& a, int m) {  // m / G
  return a.G == 1 ? m : (int)__umulhi((unsigned)m, a.g_inv);
}

// The last CTA of a grid has no tiles: it checks the sequences (tree and
// pages; slot, length and count come from seq_info) and writes their plans
// and status, while the others work.  One warp per sequence.
template <int THREADS>
__device__ __forceinline__ void check_sequences(const TreeArgs& a, int rows, int tile_shift, int n_cta,
                                                long long* s_part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long total = 0, chunk = 0;
  for (int base = 0; base < a.n_seq; base += THREADS) {
    block_excl<THREADS>(base + tid < a.n_seq ? seq_info(a, base + tid, rows, tile_shift).work() : 0, s_part,
                        &chunk);
    total += chunk;
  }
  const long long share = max(share_of(total, n_cta), 1ll);
  long long first = 0;
  for (int base = 0; base < a.n_seq; base += THREADS) {
    SeqInfo q;
    if (base + tid < a.n_seq) q = seq_info(a, base + tid, rows, tile_shift);
    const long long excl = block_excl<THREADS>(base + tid < a.n_seq ? q.work() : 0, s_part, &chunk);
    if (base + tid < a.n_seq) {
      TreePlan p;
      p.before = first + excl;
      p.share = share;
      p.tiles = q.tiles;
      p.nodes = p.status = p.pad = 0;  // by the warp that checks
      a.plan[base + tid] = p;
    }
    first += chunk;
  }
  __syncthreads();
  for (int s = warp; s < a.n_seq; s += THREADS / 32) {
    const SeqInfo q = seq_info(a, s, rows, tile_shift);
    int st = q.bad;
    if (st == 0) {
      bool bad = false;
      if (a.parents != nullptr)
        for (int i = lane; i < q.m; i += 32) {
          const int p = a.parents[(int64_t)s * a.nt + i];
          bad |= p < -1 || p >= i;
        }
      if (__any_sync(0xffffffffu, bad)) st |= SPEC_ST_TREE;
      const int held = q.m == 0 || q.len == 0 ? 0 : (q.len - 1) / a.page_size + 1;
      // with a window, the pages between the sinks and the window may be gone
      const int e1 = q.sinks > 0 ? (q.sinks - 1) / a.page_size + 1 : 0;
      const int e0 = q.lo < q.len ? q.lo / a.page_size : held;
      bad = false;
      for (int e = lane; e < held; e += 32) {
        if (e >= e1 && e < e0) continue;
        const int p = a.table[(int64_t)q.slot * a.max_pages + e];
        bad |= p < 0 || p >= a.n_pages;
      }
      if (__any_sync(0xffffffffu, bad)) st |= SPEC_ST_PAGE;
    }
    if (lane == 0) {
      a.plan[s].nodes = (st & SPEC_ST_TREE) || a.n_nodes == nullptr ? a.nt : a.n_nodes[s];
      a.plan[s].status = st;
      a.status[s] = st;
    }
  }
}

// Finds this CTA's first tile: the sequence that holds tile b * share (and
// how far into its work) goes to *at; returns its tiles' range, empty if it
// has none.
struct Range {
  long long w0, w1;
};
struct Start {
  SeqInfo q;
  long long off;
  int s;
};
template <int THREADS>
__device__ __forceinline__ Range find_range(const TreeArgs& a, int rows, int tile_shift, int n_cta,
                                            long long* s_part, Start* at) {
  long long total = 0, mine = 0, excl = 0, chunk = 0;
  const int tid = threadIdx.x;
  SeqInfo q;
  for (int base = 0; base < a.n_seq; base += THREADS) {
    mine = 0;
    if (base + tid < a.n_seq) {
      q = seq_info(a, base + tid, rows, tile_shift);
      mine = q.work();
    }
    excl = block_excl<THREADS>(mine, s_part, &chunk);
    total += chunk;
  }
  const long long share = share_of(total, n_cta);
  Range r;
  r.w0 = share * blockIdx.x;
  r.w1 = min(total, r.w0 + share);
  if (r.w0 >= r.w1) return r;
  long long first = 0;
  for (int base = 0; base < a.n_seq; base += THREADS) {
    if (a.n_seq > THREADS) {
      mine = 0;
      if (base + tid < a.n_seq) {
        q = seq_info(a, base + tid, rows, tile_shift);
        mine = q.work();
      }
      excl = block_excl<THREADS>(mine, s_part, &chunk);
    }
    if (first + excl <= r.w0 && r.w0 < first + excl + mine) {
      at->q = q;
      at->off = r.w0 - first - excl;
      at->s = base + tid;
    }
    first += chunk;
  }
  __syncthreads();
  return r;
}

// ---------------------------------------------------------------------------
// the tree of one sequence: every node's ancestors (with itself) and depth
// ---------------------------------------------------------------------------
struct TreeSmem {
  unsigned long long anc[SPEC_MAX_TREE];
  signed char depth[SPEC_MAX_TREE];
  signed char par[SPEC_MAX_TREE];
};

// Every thread of the CTA; returns whether the parents make a tree.
__device__ __forceinline__ bool load_tree(const TreeArgs& a, int s, int m, TreeSmem& t) {
  const int i = threadIdx.x;
  bool bad = false;
  __syncthreads();  // the last sequence's tree is no longer read
  if (i < SPEC_MAX_TREE) {
    int p = -1;
    if (i < m) {
      p = a.parents != nullptr ? a.parents[(int64_t)s * a.nt + i] : i - 1;
      bad = p < -1 || p >= i;
    }
    t.par[i] = (signed char)(bad ? -1 : p);
  }
  const bool any = __syncthreads_or(bad);
  if (i < m) {
    unsigned long long set = 1ull << i;
    int d = 0;
    for (int p = t.par[i]; p >= 0; p = t.par[p]) {
      set |= 1ull << p;
      d++;
    }
    t.anc[i] = set;
    t.depth[i] = (signed char)d;
  }
  __syncthreads();
  return !any;
}

}  // namespace

// The kernel for many query rows a kv head (tree_attn_tc.cu): a.rows 128 or
// 256, tiles of 128 positions, one CTA an SM.
constexpr int TREE_TC_SHIFT = 7;
cudaError_t tree_tc_launch(const TreeArgs& a, int hd, int n_cta, cudaStream_t st);
void tree_tc_init_attrs();
