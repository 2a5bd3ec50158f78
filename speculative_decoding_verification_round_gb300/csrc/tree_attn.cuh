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
  int wait_tries;      // budget of a CTA's first wait for scores (tree_set_wait_budget)
  struct TreePlan* plan;  // [n_seq]
  int32_t* status;
};

// One sequence's part of the cut, for the joining kernel.
struct TreePlan {
  long long before;  // tiles of the sequences in front of it
  long long share;   // tiles of a CTA
  int tiles;         // of each of its units
  int padded;        // and with the rest of its last piece
  int nodes;         // rows of the output that are the call's to write
  int status;
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

// The cut: CTA b takes tiles [b * share, (b + 1) * share) of the units laid
// end to end.  An even share of the total gives many CTAs the end of one unit
// and the start of the next: two pieces, each with its own first loads and its
// own end, which cost as much as about three tiles.  Where a share of up to
// three tiles more lets every CTA have one piece of one unit (the last piece
// of a unit shorter), that is taken: units count as padded to whole shares (12
// x 16 nodes over 512 positions 26.6 -> 24.8 us, 16 sequences of one node with
// a window of 4096 19.3 -> 17.8 us).
struct Cut {
  long long share;
  bool pieces;
  // tiles of a unit of q's, and with a cut into pieces the rest of its last
  __device__ __forceinline__ int padded(const SeqInfo& q) const {
    return pieces ? (int)(((unsigned)q.tiles + (unsigned)share - 1) / (unsigned)share * (unsigned)share) : q.tiles;
  }
  __device__ __forceinline__ long long work(const SeqInfo& q) const { return (long long)q.units * padded(q); }
};
constexpr int CUT_MORE = 4;   // shares that are tried: the even one, and up to three tiles more
constexpr int CUT_LONG = 64;  // from here on no share is tried
// The share, from the number of pieces that each one tried makes.
__device__ __forceinline__ Cut cut_of(long long even, const unsigned (&pieces)[CUT_MORE], int n_cta) {
  Cut c;
  c.share = even;
  c.pieces = false;
#pragma unroll
  for (int more = CUT_MORE - 1; more >= 0; more--)
    if (pieces[more] <= (unsigned)n_cta) {
      c.pieces = true;
      c.share = even + more;
    }
  return c;
}
__device__ __forceinline__ unsigned pieces_of(const SeqInfo& q, unsigned share) {
  return min((unsigned long long)q.units * (((unsigned)q.tiles + share - 1) / share), 1ull << 20);
}
__device__ __forceinline__ long long even_share(long long total, int n_cta) {
  return max(div_ll(total + n_cta - 1, n_cta), 1ll);
}

// Inclusive sum over a warp.
__device__ __forceinline__ long long warp_incl(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += y;
  }
  return v;
}

// Up to 32 sequences: every warp by itself, a lane a sequence (q: this
// lane's), without a barrier (12 x 16 nodes: 25.5 us with the barriers of the
// general form, 24.0 without).
__device__ __forceinline__ Cut cut_work_few(const TreeArgs& a, int rows, int tile_shift, int n_cta, SeqInfo& q) {
  const int lane = threadIdx.x & 31;
  q.units = 0;
  q.tiles = 1;
  if (lane < a.n_seq) q = seq_info(a, lane, rows, tile_shift);
  const long long even = even_share(__shfl_sync(0xffffffffu, warp_incl(q.work()), 31), n_cta);
  unsigned pieces[CUT_MORE];
#pragma unroll
  for (int more = 0; more < CUT_MORE; more++)
    pieces[more] = even < CUT_LONG ? __reduce_add_sync(0xffffffffu, pieces_of(q, (unsigned)even + more)) : ~0u;
  return cut_of(even, pieces, n_cta);
}

// q: this thread's sequence (with a cut into pieces there are no more of them
// than threads).  scratch: 16 bytes.
template <int THREADS>
__device__ __forceinline__ Cut cut_work(const TreeArgs& a, int rows, int tile_shift, int n_cta, long long* s_part,
                                        void* scratch, SeqInfo& q) {
  const int tid = threadIdx.x, lane = tid & 31;
  unsigned* sums = reinterpret_cast<unsigned*>(scratch);
  if (tid < CUT_MORE) sums[tid] = 0u;
  long long total = 0, chunk = 0;
  for (int base = 0; base < a.n_seq; base += THREADS) {
    long long mine = 0;
    if (base + tid < a.n_seq) {
      q = seq_info(a, base + tid, rows, tile_shift);
      mine = q.work();
    }
    block_excl<THREADS>(mine, s_part, &chunk);
    total += chunk;
  }
  const long long even = even_share(total, n_cta);
  unsigned pieces[CUT_MORE] = {~0u, ~0u, ~0u, ~0u};
  if (a.n_seq <= THREADS && even < CUT_LONG) {
#pragma unroll
    for (int more = 0; more < CUT_MORE; more++) {
      const unsigned n =
          __reduce_add_sync(0xffffffffu, tid < a.n_seq ? pieces_of(q, (unsigned)even + more) : 0u);
      if (lane == 0 && n > 0u) atomicAdd(&sums[more], n);
    }
    __syncthreads();
#pragma unroll
    for (int more = 0; more < CUT_MORE; more++) pieces[more] = sums[more];
  }
  return cut_of(even, pieces, n_cta);
}

__device__ __forceinline__ int node_of(const TreeArgs& a, int m) {  // m / G
  return a.G == 1 ? m : (int)__umulhi((unsigned)m, a.g_inv);
}

// Checks a sequence (tree and pages; slot, length and count come from
// seq_info) and writes its status.  A warp.
__device__ __forceinline__ void check_sequence(const TreeArgs& a, int s, int rows, int tile_shift) {
  const int lane = threadIdx.x & 31;
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
    const int e1 = q.sinks > 0 ? min(held, (q.sinks - 1) / a.page_size + 1) : 0;
    const int e0 = q.lo < q.len ? q.lo / a.page_size : held;
    const int32_t* row = a.table + (int64_t)q.slot * a.max_pages;
    bad = false;
    auto look = [&](int e) {
      const int p = row[e];
      bad |= p < 0 || p >= a.n_pages;
    };
#pragma unroll 4
    for (int e = lane; e < e1; e += 32) look(e);
#pragma unroll 4
    for (int e = max(e0, e1) + lane; e < held; e += 32) look(e);
    if (__any_sync(0xffffffffu, bad)) st |= SPEC_ST_PAGE;
  }
  if (lane == 0) {
    const int m = a.n_nodes != nullptr ? a.n_nodes[s] : a.nt;
    a.plan[s].nodes = m < 0 || m > a.nt ? a.nt : m;  // (q.m is 0 for a sequence in error)
    a.plan[s].status = st;
    a.status[s] = st;
  }
}

// The last CTA of a grid has no tiles: it writes the sequences' plans, while
// the others work, and checks the first of them, four a warp; those behind
// them are checked by warps of the others.
constexpr int CHECKS_A_WARP = 4;
template <int THREADS>
__device__ __forceinline__ void plan_sequences(const TreeArgs& a, int rows, int tile_shift, int n_cta,
                                               long long* s_part, void* scratch) {
  const int tid = threadIdx.x, warp = tid >> 5;
  constexpr int FIRST = CHECKS_A_WARP * (THREADS / 32);
  SeqInfo q;
  const Cut c = cut_work<THREADS>(a, rows, tile_shift, n_cta, s_part, scratch, q);
  long long first = 0, chunk = 0;
  for (int base = 0; base < a.n_seq; base += THREADS) {
    if (a.n_seq > THREADS && base + tid < a.n_seq) q = seq_info(a, base + tid, rows, tile_shift);
    const long long excl = block_excl<THREADS>(base + tid < a.n_seq ? c.work(q) : 0, s_part, &chunk);
    if (base + tid < a.n_seq) {
      TreePlan* p = a.plan + base + tid;
      p->before = first + excl;
      p->share = c.share;
      p->tiles = q.tiles;
      p->padded = c.padded(q);
    }
    first += chunk;
  }
  for (int s = warp; s < min(a.n_seq, FIRST); s += THREADS / 32) check_sequence(a, s, rows, tile_shift);
}
// The other CTAs' share of the checks, over `warps` of each.
template <int THREADS>
__device__ __forceinline__ void check_others(const TreeArgs& a, int rows, int tile_shift, int n_cta, int warps) {
  constexpr int FIRST = CHECKS_A_WARP * (THREADS / 32);
  for (long long s = FIRST + (long long)blockIdx.x * warps + (threadIdx.x >> 5); s < a.n_seq;
       s += (long long)n_cta * warps)
    check_sequence(a, (int)s, rows, tile_shift);
}

// Finds this CTA's first tile, of the sequence that holds tile b * share:
// which, and how far into its work (*at: shared memory on the way).  Returns
// how many tiles the CTA takes (0 or less: none).  What pads a unit stands
// behind its last piece, which ends there.
struct Start {
  SeqInfo q;
  long long off;
  int s, left;  // with a cut into pieces: tiles of the unit from here on
};
__device__ __forceinline__ Start start_in(const Cut& c, const SeqInfo& q, int s, long long off) {
  Start at;
  at.q = q;
  at.off = off;
  at.s = s;
  at.left = 0;
  if (c.pieces) {  // (of less than CUT_LONG + CUT_MORE tiles a CTA: 32 bits)
    const unsigned padded = (unsigned)c.padded(q), unit = (unsigned)off / padded, t0 = (unsigned)off % padded;
    at.off = unit * q.tiles + t0;
    at.left = q.tiles - (int)t0;
  }
  return at;
}
template <int THREADS>
__device__ __forceinline__ long long find_range(const TreeArgs& a, int rows, int tile_shift, int n_cta,
                                                long long* s_part, void* scratch, Start* at, Start& start) {
  const int tid = threadIdx.x;
  SeqInfo q;
  if (a.n_seq <= 32) {
    const Cut c = cut_work_few(a, rows, tile_shift, n_cta, q);
    const long long w0 = c.share * blockIdx.x, mine = c.work(q), incl = warp_incl(mine);
    const long long all = __shfl_sync(0xffffffffu, incl, 31);
    const unsigned here = __ballot_sync(0xffffffffu, incl - mine <= w0 && w0 < incl);
    if (here == 0u) return 0;
    const int src = __ffs(here) - 1;
    static_assert(sizeof(SeqInfo) % 4 == 0, "words");
    int* words = reinterpret_cast<int*>(&q);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(SeqInfo) / 4); i++) words[i] = __shfl_sync(0xffffffffu, words[i], src);
    start = start_in(c, q, src, w0 - __shfl_sync(0xffffffffu, incl - mine, src));
    const long long n = min(all, w0 + c.share) - w0;
    return c.pieces ? min(n, (long long)start.left) : n;
  }
  const Cut c = cut_work<THREADS>(a, rows, tile_shift, n_cta, s_part, scratch, q);
  const long long w0 = c.share * blockIdx.x;
  long long first = 0, chunk = 0;
  for (int base = 0; base < a.n_seq; base += THREADS) {
    if (a.n_seq > THREADS && base + tid < a.n_seq) q = seq_info(a, base + tid, rows, tile_shift);
    const long long mine = base + tid < a.n_seq ? c.work(q) : 0;
    const long long excl = block_excl<THREADS>(mine, s_part, &chunk);
    if (first + excl <= w0 && w0 < first + excl + mine) *at = start_in(c, q, base + tid, w0 - first - excl);
    first += chunk;
  }
  const long long n = min(first, w0 + c.share) - w0;
  __syncthreads();
  if (n <= 0) return 0;
  start = *at;
  return c.pieces ? min(n, (long long)start.left) : n;  // one piece, without what pads it
}

// ---------------------------------------------------------------------------
// the tree of one sequence: every node's ancestors (with itself) and depth
// ---------------------------------------------------------------------------
struct TreeSmem {
  unsigned long long anc[SPEC_MAX_TREE];
  signed char depth[SPEC_MAX_TREE];
  signed char par[SPEC_MAX_TREE];
};

// A weight goes to the MMA as hi + lo: hi is the weight cut off behind its 11th
// bit (w & P_CUT), lo = w - P_REST hi the rest and 2^-22 of hi more, so that neither is
// ever negative, and lo not 0 beside a hi that is not (down to 2^-3, where fp16
// ends): a value that is infinite stays so, where inf * 0 or inf - inf would be
// a NaN.
constexpr uint32_t P_CUT = 0xFFFFE000u;
constexpr float P_REST = 1.0f - 0x1p-22f;

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

// The kernel for many query rows a kv head (tree_attn_tc.cu): a.rows 64, 128 or
// 256, tiles of 128 positions, one CTA an SM.
constexpr int TREE_TC_SHIFT = 7;
cudaError_t tree_tc_launch(const TreeArgs& a, int hd, int n_cta, cudaStream_t st);
void tree_tc_init_attrs();
