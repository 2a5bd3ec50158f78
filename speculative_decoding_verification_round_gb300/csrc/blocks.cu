// blocks.cu -- which blocks of a cache a query attends to: digests of the
// blocks (spec_block_digest), scores from them (spec_block_scores), and the
// selection of the largest (spec_block_select).
//
// Measured: 12 prompts of 4095 positions in one layer, 8 heads of 128, blocks of 32: in 4 bits (28
// MB) 13.9 us, ten layers at a time 104: the minima and maxima of the codes' values (ALU pipe
// 60%, issue slots 59%); in fp16 (101 MB) 21, ten layers 176, 6.1 TB/s: a call of one layer is three
// blocks a warp, start and end.  Scores of their 12 x 16 nodes, 40 heads over 8, 9 us: 192
// CTAs of 64 places, of which five heads leave three of eight empty.  A decode step of 2
// sequences over 2048 blocks, digests and scores, 9.0 us in two launches.
#include <climits>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "key_warp.cuh"

namespace {

// ---------------------------------------------------------------------------
// digests: a warp per block, 16 bytes (of codes 8) a lane and load, several rows of the
// block a load, the next eight loads (of the next block, too) in flight under the
// comparisons; the lanes that hold the same channels are joined at the end, each keeping
// the half of the registers that the other one gives away
// ---------------------------------------------------------------------------
constexpr int DG_THREADS = 128, DG_WARPS = DG_THREADS / 32;

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What a digest reads: the keys' rows in fp16, or codes and scales.
struct Keys {
  const uint8_t* rows;   // fp16 rows, or codes
  const __half* scales;  // of codes
  int64_t layer_stride;  // rows
};

// REGS registers of both bounds, joined over the lanes that differ in bits [BIT, 5) of
// their number.  Afterwards a lane has REGS >> (5 - BIT) of them, from the returned
// one on: the highest lane bit chooses between the halves.
template <int REGS, int BIT>
__device__ __forceinline__ int join_lanes(uint32_t (&lo)[REGS], uint32_t (&hi)[REGS]) {
  static_assert(REGS >> (5 - BIT) > 0, "one register at least");
  const int lane = threadIdx.x & 31;
  int reg0 = 0;
#pragma unroll
  for (int bit = 4, left = REGS / 2; bit >= BIT; bit--, left /= 2) {
    const bool upper = lane >> bit & 1;
#pragma unroll
    for (int x = 0; x < REGS / 2; x++) {
      if (x >= left) break;
      const uint32_t gl = upper ? lo[x] : lo[x + left], gh = upper ? hi[x] : hi[x + left];
      const uint32_t ol = upper ? lo[x + left] : lo[x], oh = upper ? hi[x + left] : hi[x];
      lo[x] = min2(ol, __shfl_xor_sync(0xffffffffu, gl, 1 << bit));
      hi[x] = max2(oh, __shfl_xor_sync(0xffffffffu, gh, 1 << bit));
    }
    if (upper) reg0 += left;
  }
  return reg0;
}

// Blocks and pages: a division only where a page has no power of two of blocks.
struct PageBlocks {
  int shift, per, per_shift;  // log2 of the block, blocks of a page and their log2 (-1: none)
  __device__ __forceinline__ int blocks(int len) const {
    return (int)(((uint32_t)len + (1u << shift) - 1u) >> shift);  // (len is at most 2^31 - 1)
  }
  __device__ __forceinline__ int page(uint32_t b) const { return (int)(per_shift >= 0 ? b >> per_shift : b / (uint32_t)per); }
  __device__ __forceinline__ int at(uint32_t b) const { return (int)b - page(b) * per; }
};
int log2_of(int x) {  // -1: not a power of two
  int n = 0;
  while (1 << n < x && n < 30) n++;
  return 1 << n == x ? n : -1;
}
PageBlocks page_blocks(const spec_digest* dg) {
  const int per = dg->page_size / dg->block;
  return {log2_of(dg->block), per, log2_of(per)};
}

template <int HD, bool Q4>
__global__ void __launch_bounds__(DG_THREADS, Q4 ? 5 : 4)
digest_kernel(const spec_digest dg, const Keys keys, int n, const int32_t* __restrict__ slots,
              const int32_t* __restrict__ pos0, uint32_t split, const PageBlocks pb, int32_t* __restrict__ status) {
  constexpr int ROW = Q4 ? HD / 2 : HD * 2, LANES = ROW / (Q4 ? 8 : 16), PER = 32 / LANES;  // bytes; lanes and rows of a load
  constexpr int REGS = Q4 ? 8 : 4, U = 8, ROWS = U * PER;  // rows in flight
  constexpr int BIT = LANES == 16 ? 4 : LANES == 8 ? 3 : 2;
  using Load = typename std::conditional<Q4, uint2, uint4>::type;
  constexpr int KEPT = REGS >> (5 - BIT);
  grid_dep_wait();  // (nothing behind starts early: 2% less for 12 prompts)
  const int lane = threadIdx.x & 31;
  // (32 bits: the host sees to it)
  const uint32_t w = blockIdx.x * DG_WARPS + (threadIdx.x >> 5), unit = w / split, y = w - unit * split;
  const uint32_t il = unit / dg.n_kv_heads, h = unit - il * dg.n_kv_heads, i = il / dg.n_layers, layer = il - i * dg.n_layers;
  if (i >= (uint32_t)n) return;
  const int slot = slots[i], p0 = pos0 != nullptr ? pos0[i] : 0;
  int st = 0, len = 0;
  if (slot < 0 || slot >= dg.n_slots)
    st |= SPEC_ST_SLOT;
  else
    len = dg.len[slot];
  if (p0 < 0 || len < 0 || len > dg.max_pages * dg.page_size) st |= SPEC_ST_FULL;
  const int block = dg.block, per = pb.per, nb = st == 0 ? pb.blocks(len) : 0, b0 = max(p0, 0) >> pb.shift;
  const int32_t* row = dg.table + (int64_t)(st == 0 ? slot : 0) * dg.max_pages;
  if (h == 0 && layer == 0 && y == 0) {  // the entry's status
    bool bad = false;
    if (st == 0 && b0 < nb)
      for (int e = pb.page(b0) + lane; e <= pb.page(nb - 1); e += 32) bad |= row[e] < 0 || row[e] >= dg.n_pages;
    if (__any_sync(0xffffffffu, bad)) st |= SPEC_ST_PAGE;
    if (lane == 0) status[i] = st;
  }
  const uint32_t count = nb, l = lane % LANES;
  auto page_of = [&](uint32_t b) { return b < count ? row[pb.page(b)] : -1; };
  auto rows_of = [&](uint32_t b) { return min(block, len - (int)b * block); };
  struct Part {
    Load v[U];
    uint32_t s[U];
  };
  // rows r0 ... r0 + ROWS - 1 of block b (a row again where it has no more: that changes nothing)
  auto load = [&](uint32_t b, int pg, int r0, Part& p) {
    if (b >= count || pg < 0 || pg >= dg.n_pages) return;
    const int64_t first = (int64_t)layer * keys.layer_stride + ((int64_t)pg * dg.n_kv_heads + h) * dg.page_size + pb.at(b) * block;
    const int last = rows_of(b) - 1;
    const uint8_t* src = keys.rows + first * ROW + l * (uint32_t)sizeof(Load);
    const __half* sc = Q4 ? keys.scales + first * (HD / 32) + l / 2 : nullptr;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int at = min(r0 + u * PER + lane / LANES, last);
      p.v[u] = __ldg(reinterpret_cast<const Load*>(src + at * ROW));
      if (Q4) p.s[u] = __half_as_ushort(__ldg(sc + at * (HD / 32)));
    }
  };
  uint32_t b = (uint32_t)b0 + y;
  int pg = page_of(b), pg_next = page_of(b + split), r0 = 0;
  Part now, next;
  load(b, pg, 0, now);
  uint32_t lo[REGS], hi[REGS];
  while (b < count) {
    const bool end = r0 + ROWS >= rows_of(b);
    const uint32_t b1 = end ? b + split : b;
    const int pg1 = end ? pg_next : pg, r1 = end ? 0 : r0 + ROWS;
    load(b1, pg1, r1, next);
    if (end) pg_next = page_of(b1 + split);
    if (r0 == 0) {
#pragma unroll
      for (int x = 0; x < REGS; x++) {
        lo[x] = 0x7C007C00u;
        hi[x] = 0xFC00FC00u;
      }
    }
    const int many = rows_of(b) - r0;
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (u > 0 && u * PER >= many) break;
      uint32_t q[4] = {now.v[u].x, now.v[u].y, 0u, 0u};
      if constexpr (!Q4) {
        q[2] = now.v[u].z;
        q[3] = now.v[u].w;
      }
      const uint32_t s2 = now.s[u] * 0x10001u;
#pragma unroll
      for (int x = 0; x < REGS; x++) {
        // codes: word x / 4; elements 0, 2 | 1, 3 | 16, 18 | 17, 19 of its four
        const uint32_t val = !Q4 ? q[x % 4]
                                 : kw_hmul2(x & 2 ? q4_high(q[x / 4] >> (x & 1 ? 8 : 0))
                                                  : q4_low(q[x / 4] >> (x & 1 ? 8 : 0)), s2);
        lo[x] = min2(lo[x], val);
        hi[x] = max2(hi[x], val);
      }
    }
    const uint32_t done = b;
    const int page = pg;
    now = next;
    b = b1;
    pg = pg1;
    r0 = r1;
    if (!end || page < 0 || page >= dg.n_pages) continue;
    const int64_t head = (int64_t)page * dg.n_kv_heads + h;
    const int reg0 = join_lanes<REGS, BIT>(lo, hi);
    uint16_t* to = dg.data + (int64_t)layer * dg.layer_stride + (head * per + pb.at(done)) * (2 * HD);
    if (!Q4) {  // word l * 4 + reg of the row
#pragma unroll
      for (int x = 0; x < KEPT; x++) {
        reinterpret_cast<uint32_t*>(to)[l * 4 + reg0 + x] = lo[x];
        reinterpret_cast<uint32_t*>(to + HD)[l * 4 + reg0 + x] = hi[x];
      }
    } else if (KEPT >= 2) {  // neighbours: elements 0, 2 and 1, 3 of a word's four, or 16 + ...
#pragma unroll
      for (int x = 0; x < KEPT; x += 2) {
        const int reg = reg0 + x, word = (32 * (l >> 1) + 16 * (reg >> 1 & 1) + 8 * (l & 1) + 4 * (reg >> 2)) / 2;
        *reinterpret_cast<uint2*>(reinterpret_cast<uint32_t*>(to) + word) =
            make_uint2(__byte_perm(lo[x], lo[x + 1], 0x5410), __byte_perm(lo[x], lo[x + 1], 0x7632));
        *reinterpret_cast<uint2*>(reinterpret_cast<uint32_t*>(to + HD) + word) =
            make_uint2(__byte_perm(hi[x], hi[x + 1], 0x5410), __byte_perm(hi[x], hi[x + 1], 0x7632));
      }
    } else {  // one register: elements reg & 1, + 2
      const int reg = reg0, e = 32 * (l >> 1) + 16 * (reg >> 1 & 1) + 8 * (l & 1) + 4 * (reg >> 2) + (reg & 1);
      to[e] = (uint16_t)lo[0];
      to[e + 2] = (uint16_t)(lo[0] >> 16);
      to[HD + e] = (uint16_t)hi[0];
      to[HD + e + 2] = (uint16_t)(hi[0] >> 16);
    }
  }
}

// ---------------------------------------------------------------------------
// scores: sum_d max(q lo, q hi) = min(q, 0) . lo + max(q, 0) . hi, two products with the
// digest as it lies in memory: a tile of 16 blocks a warp (its digests straight into
// the A fragments, whose order of channels the queries follow) against 8 query
// rows at a time.  A node's heads are neighbouring rows, as many as the next power of
// two (the first head again in the places behind), so that the maximum over them is taken in
// registers and by exchanges.
// ---------------------------------------------------------------------------
constexpr int SC_THREADS = 256, SC_WARPS = SC_THREADS / 32, SC_ROWS = 64;

struct ScoreArgs {
  spec_digest dg;
  int layer, n_seq, nt, nq, G, GP, gp_shift;  // GP: G to the next power of two
  const int32_t* slots;
  const int32_t* n_nodes;
  const __half* q;
  int64_t q_stride;
  float* scores;
  int64_t ld;
  int32_t* status;
  int nodes, groups;  // nodes of a CTA, CTAs for a sequence's nodes
  int chunks;         // CTAs for a sequence's blocks
  PageBlocks pb;
};

template <int HD>
__host__ __device__ constexpr int score_q_bytes(int tiles) {
  return tiles * (2 * HD / 16) * 32 * 8;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int HD>
__global__ void __launch_bounds__(SC_THREADS) scores_kernel(const ScoreArgs a) {
  constexpr int STEPS = 2 * HD / 16, LOADS = 2 * HD / 32;  // 16-byte loads of a lane and row
  extern __shared__ __align__(16) unsigned char smem[];
  grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const spec_digest& dg = a.dg;
  const int y = blockIdx.x / a.chunks, chunk = blockIdx.x - y * a.chunks, sh = y / a.groups, grp = y - sh * a.groups;
  const int s = sh / dg.n_kv_heads, h = sh - s * dg.n_kv_heads;
  const int slot = a.slots[s], m = a.n_nodes != nullptr ? a.n_nodes[s] : a.nt;
  int st = 0, len = 0;
  if (slot < 0 || slot >= dg.n_slots)
    st |= SPEC_ST_SLOT;
  else
    len = dg.len[slot];
  if (m < 0 || m > a.nt) st |= SPEC_ST_TREE;
  const int per = a.pb.per, nb = a.pb.blocks(max(len, 0));
  if (len < 0 || len > dg.max_pages * dg.page_size || nb > a.ld) st |= SPEC_ST_FULL;
  const int32_t* row = dg.table + (int64_t)(st == 0 ? slot : 0) * dg.max_pages;
  if (chunk == 0 && grp == 0 && h == 0) {
    bool bad = false;
    if (st == 0)
      for (int e = tid; nb > 0 && e <= a.pb.page(nb - 1); e += SC_THREADS) bad |= row[e] < 0 || row[e] >= dg.n_pages;
    if (__syncthreads_or(bad)) st |= SPEC_ST_PAGE;
    if (tid == 0) a.status[s] = st;
    st &= ~SPEC_ST_PAGE;
  }
  const int node0 = grp * a.nodes, nodes = min(a.nodes, m - node0), rows = nodes * a.GP;
  const int first = chunk * SC_WARPS * 16;
  if (st != 0 || nodes <= 0 || first >= nb) return;
  const int tiles = (rows + 7) / 8;
  const uint32_t qs = kw_smem(smem);
  // the digests of a tile of 16 blocks: lane (g, t) has units t, t + 4, ... of blocks g, 8 + g
  uint4 v[2][LOADS];
  bool there[2];
  auto load = [&](int b0) {
#pragma unroll
    for (int half = 0; half < 2; half++) {
      const int b = b0 + 8 * half + g, e = a.pb.page(b), pg = b < nb ? row[e] : -1;
      there[half] = pg >= 0 && pg < dg.n_pages;
      const uint4* src = reinterpret_cast<const uint4*>(
          dg.data + (int64_t)a.layer * dg.layer_stride +
          (((int64_t)(there[half] ? pg : 0) * dg.n_kv_heads + h) * per + (there[half] ? b - e * per : 0)) * (2 * HD));
#pragma unroll
      for (int i = 0; i < LOADS; i++) v[half][i] = __ldg(src + 4 * i + t);
    }
  };
  const int mine = first + warp * 16;
  if (mine < nb) load(mine);
  // the queries' fragments: 16 bytes of a row are two steps' of lo and two of hi
  constexpr int UNITS = HD / 8, IN_FLIGHT = SC_ROWS * UNITS / SC_THREADS;
  uint4 x[IN_FLIGHT];
#pragma unroll
  for (int y = 0; y < IN_FLIGHT; y++) {
    const int e = tid + y * SC_THREADS, u = e % UNITS, r = e / UNITS;
    x[y] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const int node = node0 + (r >> a.gp_shift), k = r & (a.GP - 1), head = h * a.G + (k < a.G ? k : 0);
      x[y] = *reinterpret_cast<const uint4*>(a.q + ((int64_t)s * a.nt + node) * a.q_stride + head * HD + 8 * u);
    }
  }
#pragma unroll
  for (int y = 0; y < IN_FLIGHT; y++) {
    const int e = tid + y * SC_THREADS, u = e % UNITS, r = e / UNITS, i = u >> 2, col = r & 7, n = r >> 3;
    if (n >= tiles) break;
    const uint32_t to = qs + ((n * STEPS + 2 * i) * 32 + col * 4 + (u & 3)) * 8;
    kw_sts64(to, min2(x[y].x, 0u), min2(x[y].y, 0u));
    kw_sts64(to + 256, min2(x[y].z, 0u), min2(x[y].w, 0u));
    kw_sts64(to + STEPS * 128, max2(x[y].x, 0u), max2(x[y].y, 0u));
    kw_sts64(to + STEPS * 128 + 256, max2(x[y].z, 0u), max2(x[y].w, 0u));
  }
  __syncthreads();
  const int64_t out0 = (((int64_t)s * a.nt + node0) * dg.n_kv_heads + h) * a.ld, node_ld = (int64_t)dg.n_kv_heads * a.ld;
  for (int b0 = mine; b0 < nb; b0 += a.chunks * SC_WARPS * 16) {
    if (b0 != mine) load(b0);
    float top[2];  // of a node with more than 8 heads
    auto put = [&](int node, int half, float value) {
      const int b = b0 + 8 * half + g;
      if (b < nb && node < nodes) a.scores[out0 + node * node_ld + b] = value;
    };
    for (int n0 = 0; n0 < tiles; n0 += 2) {  // two tiles' products, four sums, at a time
      float sum[2][2][4];
#pragma unroll
      for (int z = 0; z < 2; z++)
#pragma unroll
        for (int e = 0; e < 4; e++) sum[z][0][e] = sum[z][1][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < LOADS / 2; i++) {
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const uint4 &l0 = v[0][i], &l1 = v[1][i], &h0 = v[0][i + LOADS / 2], &h1 = v[1][i + LOADS / 2];
          const uint32_t al[4] = {k ? l0.z : l0.x, k ? l1.z : l1.x, k ? l0.w : l0.y, k ? l1.w : l1.y};
          const uint32_t ah[4] = {k ? h0.z : h0.x, k ? h1.z : h1.x, k ? h0.w : h0.y, k ? h1.w : h1.y};
#pragma unroll
          for (int z = 0; z < 2; z++) {
            // (the last of an odd number twice)
            const uint32_t at = qs + ((min(n0 + z, tiles - 1) * STEPS + 2 * i + k) * 32 + lane) * 8;
            const uint2 ql = kw_lds64(at), qh = kw_lds64(at + STEPS * 128);
            mma_16816(sum[z][0], al, ql.x, ql.y);
            mma_16816(sum[z][1], ah, qh.x, qh.y);
          }
        }
      }
#pragma unroll
      for (int z = 0; z < 2; z++) {
        const int n = n0 + z;
        if (n >= tiles) break;
        // (block g, rows 2t, 2t + 1), (block 8 + g, ...)
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = there[e >> 1] ? sum[z][0][e] + sum[z][1][e] : -INFINITY;
        if (a.GP == 1) {
#pragma unroll
          for (int e = 0; e < 4; e++) put(8 * n + 2 * t + (e & 1), e >> 1, x[e]);
        } else {
          float y[2] = {max_nan(x[0], x[1]), max_nan(x[2], x[3])};
          if (a.GP >= 4)
#pragma unroll
            for (int e = 0; e < 2; e++) y[e] = max_nan(y[e], __shfl_xor_sync(0xffffffffu, y[e], 1));
          if (a.GP >= 8)
#pragma unroll
            for (int e = 0; e < 2; e++) y[e] = max_nan(y[e], __shfl_xor_sync(0xffffffffu, y[e], 2));
          if (a.GP <= 8) {
            const int shift = a.gp_shift - 1;  // lanes t of a node
            if ((t & ((1 << shift) - 1)) == 0)
#pragma unroll
              for (int e = 0; e < 2; e++) put((4 >> shift) * n + (t >> shift), e, y[e]);
          } else {
            const int part = n & (a.GP / 8 - 1);
#pragma unroll
            for (int e = 0; e < 2; e++) top[e] = part == 0 ? y[e] : max_nan(top[e], y[e]);
            if (part == a.GP / 8 - 1 && t == 0)
#pragma unroll
              for (int e = 0; e < 2; e++) put(n >> (a.gp_shift - 3), e, top[e]);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// selection: a CTA per row, a row's keys (its scores as whole numbers in the same
// order) in registers, neighbours in neighbouring lanes.  The k-th largest key lies in a
// bin of a histogram of the ten highest bits in which the row's keys differ; of the
// bin's keys, mostly a few, each is ranked against the others (192 x 8 rows of 2048: 15
// us with the k-th key's bits found one by one by counts, 13 with eight bits, whose bins
// most keys share; 10.2 so with ten CTAs an SM, 10.5 with nine, 11.4 with eleven, for
// which registers are spilled).  A warp's vote over a key of each lane is a word of the
// map of the chosen blocks, whose words then are written out in order, a thread one.
// ---------------------------------------------------------------------------
struct SelectArgs {
  const int32_t* len;
  int n_slots, shift, n_seq, nt, nkv;  // shift: log2 of the block
  const int32_t* slots;
  const int32_t* n_nodes;
  const float* scores;
  int64_t ld;
  int keep, first, last;
  int32_t* blocks;
  int32_t* status;
};

template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS, THREADS == 128 && PER == 16 ? 10 : 1) select_kernel(const SelectArgs a) {
  constexpr int WARPS = THREADS / 32, SPAN = THREADS * PER, CAND = 256, WORDS = SPAN / 32;
  constexpr int BIN_BITS = THREADS <= 64 ? 9 : 10, BINS = 1 << BIN_BITS, EACH = BINS / THREADS;
  static_assert(WORDS <= THREADS && PER <= 32, "a word a thread, a lane for each of a thread's keys");
  __shared__ int s_sum[2][WARPS], s_n, s_found[3];
  __shared__ __align__(16) uint32_t s_hist[BINS];
  __shared__ uint32_t s_bits[2][WORDS], s_mm[2][WARPS], s_cand[CAND], s_key;
  grid_dep_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x, sn = r / a.nkv, h = r - sn * a.nkv, s = sn / a.nt, node = sn - s * a.nt;
  const int slot = a.slots[s], m = a.n_nodes != nullptr ? a.n_nodes[s] : a.nt;
  int st = 0, len = 0;
  if (slot < 0 || slot >= a.n_slots)
    st |= SPEC_ST_SLOT;
  else
    len = a.len[slot];
  if (m < 0 || m > a.nt) st |= SPEC_ST_TREE;
  const int nb = (int)(((uint32_t)max(len, 0) + (1u << a.shift) - 1u) >> a.shift);
  if (len < 0 || nb > a.ld) st |= SPEC_ST_FULL;
  if (h == 0 && node == 0 && tid == 0) a.status[s] = st;
  int32_t* out = a.blocks + (int64_t)r * a.keep;
  if ((st & SPEC_ST_TREE) == 0 && node >= m) return;
  const int k = st != 0 ? 0 : min(nb, a.keep);
  for (int j = k + tid; j < a.keep; j += THREADS) out[j] = -1;
  if (k == nb || st != 0) {
    for (int j = tid; j < k; j += THREADS) out[j] = j;
    return;
  }
  // Of the blocks [a.first, nb - a.last) `need` are chosen, the others are.  A key is
  // never 0, which stands for no block.
  const float* x = a.scores + (int64_t)r * a.ld;
  const int end = nb - a.last, need = k - a.first - a.last;
  const uint32_t many = (uint32_t)max(end - a.first, 0);
  const bool one = nb <= SPAN;
  uint32_t key[PER];
  auto load = [&](int c0) {  // key i: block c0 + i THREADS + tid
    float f[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int j = c0 + i * THREADS + tid;
      f[i] = (uint32_t)(j - a.first) < many ? x[j] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int j = c0 + i * THREADS + tid;
      key[i] = (uint32_t)(j - a.first) < many ? (f[i] != f[i] ? 0xFF800000u : logit_key(f[i])) : 0u;
    }
  };
  // f of every key of the row but 0 (longer rows are read again for each use)
  auto each_key = [&](auto&& f) {
    for (int c0 = 0; c0 < nb; c0 += SPAN) {
      if (!one) load(c0);
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (key[i] != 0u) f(key[i]);
    }
  };
  int which = 0;
  auto count = [&](uint32_t t) {  // keys >= t > 0
    int c = 0;
    each_key([&](uint32_t y) { c += y >= t; });
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) s_sum[which][warp] = c;
    __syncthreads();
    c = __reduce_add_sync(0xffffffffu, lane < WARPS ? s_sum[which][lane] : 0);
    which ^= 1;
    return c;
  };
  // exclusive sum over the CTA's threads; *all: the whole
  auto scan = [&](int v, int* all) {
    int at = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, at, off);
      if (lane >= off) at += z;
    }
    int total = __shfl_sync(0xffffffffu, at, 31), before = at - v;
    if (WARPS > 1) {
      __syncthreads();
      if (lane == 31) s_sum[0][warp] = at;
      __syncthreads();
      total = 0;
#pragma unroll 4
      for (int w = 0; w < WARPS; w++) {
        const int c = s_sum[0][w];
        if (w < warp) before += c;
        total += c;
      }
    }
    *all = total;
    return before;
  };
  load(0);
  for (int b = tid; b < BINS; b += THREADS) s_hist[b] = 0u;
  if (tid == 0) s_n = 0;
  // the bits that all keys have in common
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
  each_key([&](uint32_t y) {
    hi = max(hi, y);
    lo = min(lo, y);
  });
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 0) {
    s_mm[0][warp] = hi;
    s_mm[1][warp] = lo;
  }
  __syncthreads();
  hi = __reduce_max_sync(0xffffffffu, lane < WARPS ? s_mm[0][lane] : 0u);
  lo = __reduce_min_sync(0xffffffffu, lane < WARPS ? s_mm[1][lane] : 0xFFFFFFFFu);
  // t: the largest number that `need` keys reach (above all keys if none is needed); reach: how
  // many do
  uint32_t t = need > 0 ? lo : 0xFFFFFFFFu;
  int reach = need > 0 ? end - a.first : 0;
  if (need > 0 && hi != lo) {
    const int top = 31 - __clz((int)(hi ^ lo)), shift = max(0, top - (BIN_BITS - 1));
    const uint32_t bins = 2u << (top - shift);
    t = hi & ~((2u << top) - 1u);
    // bins from the highest on
    each_key([&](uint32_t y) { atomicAdd(&s_hist[~(y >> shift) & (bins - 1u)], 1u); });
    __syncthreads();
    // EACH bins a thread
    using Some = typename std::conditional<EACH % 4 == 0, int4, typename std::conditional<EACH == 2, int2, int>::type>::type;
    constexpr int EVERY = sizeof(Some) / 4;
    __align__(16) int c[EACH];
    int mine = 0, all;
#pragma unroll
    for (int i = 0; i < EACH; i += EVERY)
      *reinterpret_cast<Some*>(c + i) = *reinterpret_cast<const Some*>(s_hist + EACH * tid + i);
#pragma unroll
    for (int i = 0; i < EACH; i++) mine += c[i];
    int over = scan(mine, &all);
    if (over < need && need <= over + mine) {
#pragma unroll
      for (int i = 0; i < EACH; i++) {
        if (over < need && need <= over + c[i]) {
          s_found[0] = EACH * tid + i;
          s_found[1] = over;
          s_found[2] = c[i];
        }
        over += c[i];
      }
    }
    __syncthreads();
    const uint32_t bin = bins - 1u - (uint32_t)s_found[0];
    const int above = s_found[1], in_bin = s_found[2], rest = need - above;
    t |= bin << shift;
    reach = above + in_bin;
    if (reach != need && shift > 0) {
      if (in_bin <= CAND) {
        each_key([&](uint32_t y) {
          if (((y >> shift) & (bins - 1u)) == bin) s_cand[atomicAdd(&s_n, 1)] = y;
        });
        __syncthreads();
        for (int e = tid; e < in_bin; e += THREADS) {
          const uint32_t y = s_cand[e];
          int more = 0, same = 0;
          for (int z = 0; z < in_bin; z++) {
            more += s_cand[z] > y;
            same += s_cand[z] == y;
          }
          if (more < rest && rest <= more + same) {  // (several of the same key)
            s_key = y;
            s_found[0] = above + more + same;
          }
        }
        __syncthreads();
        t = s_key;
        reach = s_found[0];
      } else {  // bit by bit
        for (uint32_t bit = 1u << (shift - 1); bit != 0u && reach != need; bit >>= 1) {
          const int c = count(t | bit);
          if (c >= need) {
            t |= bit;
            reach = c;
          }
        }
      }
    }
  }
  // Where more reach it than are needed, the search has come to its end: t is a key, and
  // of the equal ones the lowest blocks are taken.
  const int ties = reach > need ? need - count(t + 1u) : 0;
  const bool tied = reach > need;
  int base = 0, ties_before = 0;
  for (int c0 = 0; c0 < nb; c0 += SPAN) {
    if (!one) load(c0);
    // a vote a key: blocks c0 + i THREADS + 32 warp ... + 31; lane i keeps the word
    uint32_t word = 0u, equal = 0u;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const uint32_t v = __ballot_sync(0xffffffffu, need > 0 && key[i] >= t);
      if (lane == i) word = v;
    }
    if (tied)
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const uint32_t v = __ballot_sync(0xffffffffu, key[i] == t);
        if (lane == i) equal = v;
      }
    if (lane < PER) {
      s_bits[0][lane * WARPS + warp] = word & ~equal;
      s_bits[1][lane * WARPS + warp] = equal;
    }
    __syncthreads();
    uint32_t w = 0u;
    if (tid < WORDS) {
      w = s_bits[0][tid];
      equal = s_bits[1][tid];
      // the first and the last ones
      const int j0 = c0 + 32 * tid;
      auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
      w |= below(a.first - j0) | (below(nb - j0) & ~below(end - j0));
    }
    int all;
    if (tied) {
      const int before = ties_before + scan(tid < WORDS ? __popc(equal) : 0, &all);
      if (tid < WORDS)
        for (int left = ties - before; left > 0 && equal != 0u; left--, equal &= equal - 1u) w |= equal & -equal;
      ties_before += all;
    }
    int at = base + scan(__popc(w), &all);
    base += all;
    for (; w != 0u; w &= w - 1u) out[at++] = c0 + tid * 32 + __ffs(w) - 1;
    __syncthreads();  // the map has been read
  }
}

int check_digest(const spec_digest* dg) {
  if (dg == nullptr || dg->data == nullptr || dg->table == nullptr || dg->len == nullptr)
    return fail(SPEC_E_INVALID, "null digest, table or len");
  if (dg->n_layers < 1 || dg->n_pages < 1 || dg->n_kv_heads < 1 || dg->page_size < 1 || dg->n_slots < 1 ||
      dg->max_pages < 1)
    return fail(SPEC_E_SHAPE, "bad digest dimensions");
  if (dg->head_dim != 64 && dg->head_dim != 128)
    return fail(SPEC_E_UNSUPPORTED, "digests support head_dim 64 or 128");
  if (!block_fits(dg->block, dg->page_size))
    return fail(SPEC_E_SHAPE, "block must be 16, 32, 64 or 128 and divide page_size");
  if ((reinterpret_cast<uintptr_t>(dg->data) & 15u) != 0) return fail(SPEC_E_SHAPE, "data must be 16-byte aligned");
  if ((int64_t)dg->max_pages * dg->page_size > INT32_MAX)
    return fail(SPEC_E_SHAPE, "max_pages * page_size must stay below 2^31 positions");
  const double elems = (double)dg->n_pages * dg->n_kv_heads * dg->page_size * dg->head_dim;
  if (elems > 4.0e15) return fail(SPEC_E_SHAPE, "a layer's digests are too large");
  const int64_t layer = (int64_t)dg->n_pages * dg->n_kv_heads * (dg->page_size / dg->block) * 2 * dg->head_dim;
  if (dg->layer_stride % 8 != 0 || (dg->n_layers > 1 && dg->layer_stride < layer) ||
      (double)dg->layer_stride * dg->n_layers > 4.0e15)
    return fail(SPEC_E_SHAPE, "layer_stride must be a multiple of 8 and hold a layer's digests");
  return SPEC_OK;
}

int launch_digest(const spec_digest* dg, const Keys& keys, bool q4, int n, const int32_t* slots, const int32_t* pos0,
                  int32_t* status, void* stream) {
  if (slots == nullptr || status == nullptr) return fail(SPEC_E_INVALID, "null argument");
  if (n < 1) return fail(SPEC_E_SHAPE, "n >= 1 required");
  const double units = (double)n * dg->n_layers * dg->n_kv_heads;
  if (units > (1 << 30)) return fail(SPEC_E_SHAPE, "n * n_layers * n_kv_heads too large");
  // warps of a unit: two waves of what is resident, where the blocks are that many (12 prompts
  // of 4095 in 4 bits are 4% faster with three waves, 4% slower with one; a step's new blocks of 2
  // sequences, for which most warps have nothing to do, with their scores 9.6, 8.9 and 8.4 us)
  const int64_t most = (int64_t)dg->max_pages * (dg->page_size / dg->block);
  const int64_t fit = std::max<int64_t>(1, std::min<int64_t>(most, (int64_t)(device_sms() * 40 / units)));
  const int64_t rounds = (most + fit - 1) / fit;
  const int split = (int)((most + rounds - 1) / rounds);
  const size_t grid = (size_t)((units * split + DG_WARPS - 1) / DG_WARPS);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto kernel = dg->head_dim == 128 ? (q4 ? digest_kernel<128, true> : digest_kernel<128, false>)
                                    : (q4 ? digest_kernel<64, true> : digest_kernel<64, false>);
  const cudaError_t e = launch_dependent(kernel, grid, DG_THREADS, 0, st, *dg, keys, n, slots, pos0, (uint32_t)split,
                                         page_blocks(dg), status);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("block digest: ") + cudaGetErrorString(e));
  return SPEC_OK;
}

}  // namespace

bool block_fits(int block, int page_size) {
  return (block == 16 || block == 32 || block == 64 || block == 128) && page_size % block == 0;
}

static_assert(score_q_bytes<128>(SC_ROWS / 8) <= 48 * 1024, "without an attribute of the kernel's");

static bool same_sizes(const spec_digest* dg, int n_layers, int n_pages, int nkv, int page, int hd) {
  return dg->n_layers == n_layers && dg->n_pages == n_pages && dg->n_kv_heads == nkv && dg->page_size == page &&
         dg->head_dim == hd;
}

extern "C" int spec_block_digest(const spec_digest* dg, const spec_pages* kv, int n, const int32_t* slots,
                                 const int32_t* pos0, int32_t* status, void* stream) {
  int rc = check_digest(dg);
  if (rc == SPEC_OK) rc = check_pages(kv, false);
  if (rc != SPEC_OK) return rc;
  if (!same_sizes(dg, kv->n_layers, kv->n_pages, kv->n_kv_heads, kv->page_size, kv->head_dim))
    return fail(SPEC_E_SHAPE, "the digest's sizes are not the cache's");
  if (kv->layer_stride % kv->head_dim != 0) return fail(SPEC_E_SHAPE, "the cache's layer stride must be whole rows");
  const Keys keys = {reinterpret_cast<const uint8_t*>(kv->k), nullptr, kv->layer_stride / kv->head_dim};
  return launch_digest(dg, keys, false, n, slots, pos0, status, stream);
}

extern "C" int spec_block_digest_q4(const spec_digest* dg, const spec_pages_q4* kv, int n, const int32_t* slots,
                                    const int32_t* pos0, int32_t* status, void* stream) {
  int rc = check_digest(dg);
  if (rc == SPEC_OK) rc = check_pages_q4(kv, false);
  if (rc != SPEC_OK) return rc;
  if (!same_sizes(dg, kv->n_layers, kv->n_pages, kv->n_kv_heads, kv->page_size, kv->head_dim))
    return fail(SPEC_E_SHAPE, "the digest's sizes are not the cache's");
  const Keys keys = {kv->k_qs, reinterpret_cast<const __half*>(kv->k_scales), kv->layer_stride};
  return launch_digest(dg, keys, true, n, slots, pos0, status, stream);
}

extern "C" int spec_block_scores(const spec_digest* dg, int layer, int n_seq, const int32_t* slots, int nt,
                                 const int32_t* n_nodes, int n_q_heads, const uint16_t* q, int64_t q_stride,
                                 float* scores, int64_t ld, int32_t* status, void* stream) {
  const int rc = check_digest(dg);
  if (rc != SPEC_OK) return rc;
  if (slots == nullptr || q == nullptr || scores == nullptr || status == nullptr)
    return fail(SPEC_E_INVALID, "null argument");
  if (layer < 0 || layer >= dg->n_layers) return fail(SPEC_E_SHAPE, "layer out of range");
  if (n_seq < 1 || nt < 1 || nt > SPEC_MAX_TREE) return fail(SPEC_E_SHAPE, "n_seq >= 1 and nt in [1, 64] required");
  if (n_q_heads < 1 || n_q_heads % dg->n_kv_heads != 0)
    return fail(SPEC_E_SHAPE, "n_q_heads must be a positive multiple of n_kv_heads");
  if (n_q_heads / dg->n_kv_heads > SC_ROWS) return fail(SPEC_E_UNSUPPORTED, "more than 64 query heads a kv head");
  if (((reinterpret_cast<uintptr_t>(q) & 15u) | (reinterpret_cast<uintptr_t>(scores) & 3u)) != 0)
    return fail(SPEC_E_SHAPE, "q must be 16-byte aligned, scores 4-byte aligned");
  const int64_t row = (int64_t)n_q_heads * dg->head_dim;
  if (q_stride == 0) q_stride = row;
  if (q_stride % 8 != 0 || q_stride < row || (double)q_stride * n_seq * nt > 4.0e15)
    return fail(SPEC_E_SHAPE, "q_stride must be a multiple of 8 that holds a row's heads");
  if (ld < 1 || ld > (1ll << 31) || (double)ld * n_seq * nt * dg->n_kv_heads > 4.0e15)
    return fail(SPEC_E_SHAPE, "ld outside [1, 2^31], or scores too large");
  ScoreArgs a;
  a.dg = *dg;
  a.pb = page_blocks(dg);
  a.layer = layer;
  a.n_seq = n_seq;
  a.nt = nt;
  a.nq = n_q_heads;
  a.G = n_q_heads / dg->n_kv_heads;
  a.slots = slots;
  a.n_nodes = n_nodes;
  a.q = reinterpret_cast<const __half*>(q);
  a.q_stride = q_stride;
  a.scores = scores;
  a.ld = ld;
  a.status = status;
  a.gp_shift = 0;
  while (1 << a.gp_shift < a.G) a.gp_shift++;
  a.GP = 1 << a.gp_shift;
  a.nodes = std::min(nt, SC_ROWS / a.GP);
  a.groups = (nt + a.nodes - 1) / a.nodes;
  // a tile of 16 blocks a warp, until there are CTAs for eight an SM
  const int64_t most = std::min<int64_t>(ld, (int64_t)dg->max_pages * (dg->page_size / dg->block));
  const double units = (double)n_seq * dg->n_kv_heads * a.groups;
  const int64_t fill = std::max<int64_t>(1, (int64_t)(8 * device_sms() / units));
  a.chunks = (int)std::min<int64_t>((most + 16 * SC_WARPS - 1) / (16 * SC_WARPS), fill);
  if (units * a.chunks > INT32_MAX) return fail(SPEC_E_SHAPE, "n_seq * nt * n_kv_heads too large");
  const int tiles = (a.nodes * a.GP + 7) / 8;
  const size_t smem = dg->head_dim == 128 ? score_q_bytes<128>(tiles) : score_q_bytes<64>(tiles);
  const cudaError_t e =
      launch_dependent(dg->head_dim == 128 ? scores_kernel<128> : scores_kernel<64>, (size_t)(units * a.chunks),
                       SC_THREADS, smem, reinterpret_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("block scores: ") + cudaGetErrorString(e));
  return SPEC_OK;
}

extern "C" int spec_block_select(const int32_t* len, int n_slots, int block, int n_seq, const int32_t* slots, int nt,
                                 const int32_t* n_nodes, int n_kv_heads, const float* scores, int64_t ld, int n_keep,
                                 int n_first, int n_last, int32_t* blocks, int32_t* status, void* stream) {
  if (len == nullptr || slots == nullptr || scores == nullptr || blocks == nullptr || status == nullptr)
    return fail(SPEC_E_INVALID, "null argument");
  if (n_slots < 1 || n_kv_heads < 1 || n_seq < 1 || nt < 1 || nt > SPEC_MAX_TREE)
    return fail(SPEC_E_SHAPE, "n_slots, n_kv_heads and n_seq >= 1 and nt in [1, 64] required");
  if (!block_fits(block, block)) return fail(SPEC_E_SHAPE, "block must be 16, 32, 64 or 128");
  if (n_keep < 1 || n_keep > SPEC_MAX_KEEP || n_first < 0 || n_last < 0 || (int64_t)n_first + n_last > n_keep)
    return fail(SPEC_E_SHAPE, "n_keep in [1, 4096] and 0 <= n_first + n_last <= n_keep required");
  if (((reinterpret_cast<uintptr_t>(scores) | reinterpret_cast<uintptr_t>(blocks)) & 3u) != 0)
    return fail(SPEC_E_SHAPE, "scores and blocks must be 4-byte aligned");
  const double rows = (double)n_seq * nt * n_kv_heads;
  if (rows > INT32_MAX || ld < 1 || ld > (1ll << 31) || rows * ld > 4.0e15)
    return fail(SPEC_E_SHAPE, "n_seq * nt * n_kv_heads or ld too large");
  const SelectArgs a = {len, n_slots, log2_of(block), n_seq, nt, n_kv_heads, slots, n_nodes, scores, ld, n_keep, n_first,
                        n_last, blocks, status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t grid = (size_t)rows;
  // 16 keys a thread (1536 rows of 2048: with 32 2% slower, with 64 47%, with 8 28%), up to
  // 16384 a row (longer ones are read again for each use); for no more rows than SMs, each
  // with an SM to itself, 4 (8 rows of 500 3.3 us, with 8 3.8, with 16 4.9) or 8 (of 2048 3.8, 3.7,
  // 4.4; of 4096 5.8, 4.3, 4.5; of 8192 with 8 7.2, with 16 5.7).  The host knows no row's length, but no row has more blocks than ld.
  const bool few = rows <= device_sms() && ld <= 4096;
  const cudaError_t e = few ? (ld <= 512    ? launch_dependent(select_kernel<128, 4>, grid, 128, 0, st, a)
                               : ld <= 1024 ? launch_dependent(select_kernel<256, 4>, grid, 256, 0, st, a)
                               : ld <= 2048 ? launch_dependent(select_kernel<256, 8>, grid, 256, 0, st, a)
                                            : launch_dependent(select_kernel<512, 8>, grid, 512, 0, st, a))
                        : ld <= 512  ? launch_dependent(select_kernel<32, 16>, grid, 32, 0, st, a)
                        : ld <= 1024 ? launch_dependent(select_kernel<64, 16>, grid, 64, 0, st, a)
                        : ld <= 2048 ? launch_dependent(select_kernel<128, 16>, grid, 128, 0, st, a)
                        : ld <= 4096 ? launch_dependent(select_kernel<256, 16>, grid, 256, 0, st, a)
                        : ld <= 8192 ? launch_dependent(select_kernel<512, 16>, grid, 512, 0, st, a)
                                     : launch_dependent(select_kernel<1024, 16>, grid, 1024, 0, st, a);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("block selection: ") + cudaGetErrorString(e));
  return SPEC_OK;
}
