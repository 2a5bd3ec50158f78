// q4_attn.cu -- tree attention over a cache held in 4 bits (spec_tree_attn_q4).
//
// The units, their cut over the CTAs, the trees and the joining kernel are
// those of the cache in fp16 (tree_attn.cuh, tree_attn.cu); the tree's own
// nodes are fp16 here, too.  The kernel streams the codes and scales as they
// are, 0.28 of the bytes of fp16, and makes the operands of the products
// in registers (key_warp.cuh): a tile of fp16 in shared memory between would
// be written and read once, 8 cycles of the SM's shared memory a position of
// 128 dimensions where the HBM delivers one in 6.
//
// Measured (32 heads over 8 of 128): 4 x 4 nodes over 131071 positions (604 MB) 197 us, 3.1
// TB/s; with one node (4 rows a kv head) over 65536 82 us, 3.7 TB/s.  The loads alone
// run at 5.4 TB/s; what bounds it is a warp's chain of codes to operands, products and
// weights, about 24 instructions a position of 8 rows, with 12 to 16 warps an SM (issue
// slots 51% used, the tensor pipe 45%).  Other stages, CTAs an SM and keys at a time are up to
// 12% slower.  One node over 8191 positions 12.3 us: a tile of 128 a CTA, 520 of them, whose 65
// results a unit a second kernel joins; 16 sequences in a window of 4096 (14 heads over 2
// of 64) 11.3: four CTAs a unit, one an SM, 131 steps of 32 positions over their 32 warps,
// four or five each.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "key_warp.cuh"
#include "tree_attn.cuh"

namespace {

// ---------------------------------------------------------------------------
// Every warp has 32 positions of a tile of 128 and a ring of its own for them,
// so that no barrier stands between the tiles; the four warps' results are
// joined at the end of a piece.
// ---------------------------------------------------------------------------
constexpr int QA_SHIFT = 7, QA_KEYS = 1 << QA_SHIFT, QA_THREADS = 128, QA_WARPS = 4, WARP_KEYS = 32;

template <int HD, int NT>
struct QShape {
  static constexpr int ROWS = 8 * NT;
  static constexpr int STAGES = 2;
  static constexpr int CODES = WARP_KEYS * HD / 2, SCALES = WARP_KEYS * HD / 16;
  static constexpr int STAGE = 2 * (CODES + SCALES);  // bytes: K's and V's codes, K's and V's scales
  static constexpr int RING = STAGES * STAGE;         // of a warp
  using Join = JoinShape<HD, ROWS, QA_WARPS>;
  static constexpr int XROW = Join::XROW;
  static constexpr int NODES = NT == 4 ? 32 : 16;     // rows of the tree's own tile (no more nodes than rows)
  static constexpr int TREE_OFF = ((QA_WARPS * RING > Join::EXCHANGE ? QA_WARPS * RING : Join::EXCHANGE) + 127) / 128 * 128;
  static constexpr int Q_OFF = TREE_OFF + 2 * NODES * HD * 2;
  static constexpr int SUM_OFF = Q_OFF + KeyWarp<HD, NT, true>::Q_BYTES;
  static constexpr int END = SUM_OFF + KeyWarp<HD, NT, true>::SUM_BYTES;
  static constexpr size_t SMEM = END;
  // (with fewer registers a thread and more CTAs a warp has less under way at a time: 16 rows of 64
  // dimensions 122 us with three, 130 with five; of 128 108 with three, 121 with four)
  static constexpr int RESIDENT = NT == 4 ? 2 : HD == 64 ? (NT == 2 ? 3 : 4) : NT == 2 ? 3 : 4;
};

// What a unit's rows see.
template <int HD, int NT>
struct UnitRows {
  const TreeArgs& a;
  const TreeSmem& tree;
  int len, row0, M;
  // bits of the keys (g, 8 + g, ...) of 32 positions from `base` on that row r
  // sees, or of 16 nodes from `base` on
  __device__ __forceinline__ uint32_t visible(bool nodes, int base, int r, int gk) const {
    const int m = row0 + r, node = m < M ? node_of(a, m) : 0;
    const int pos = len + tree.depth[node];
    const unsigned long long anc = m < M ? tree.anc[node] : 0ull;
    uint32_t bits = 0u;
    const int count = nodes ? 2 : WARP_KEYS / 8;
#pragma unroll
    for (int i = 0; i < WARP_KEYS / 8; i++) {
      if (i >= count) break;
      const int key = base + 8 * i + gk;
      bool see;
      int p = key;
      if (nodes) {
        see = (anc >> key) & 1;
        p = len + (see ? tree.depth[key] : 0);
      } else {
        see = key < len;
      }
      if (a.window > 0) see = see && (p < a.sinks || p > pos - a.window);
      bits |= (uint32_t)see << i;
    }
    return bits;
  }
};

// 32 positions from `base` on, in a stage of the warp's ring.
template <int HD, int NT>
__device__ __forceinline__ void step_codes(KeyWarp<HD, NT, true>& kw, const UnitRows<HD, NT>& rows, uint32_t ks,
                                           uint32_t qs, uint32_t sums, float scale, int base, bool masked) {
  using Sh = QShape<HD, NT>;
  constexpr int KT = NT == 4 ? 1 : 2;  // tiles of 16 keys at a time
  const uint32_t vs = ks + Sh::CODES, kss = vs + Sh::CODES, vss = kss + Sh::SCALES;
  const int lane = threadIdx.x & 31, gk = kw.g;
  bool odd = false;
  if (masked)  // this lane's position's scales
#pragma unroll
    for (int b = 0; b < HD / 32; b++) odd |= odd_scale(kw_lds16(vss + lane * (HD / 16) + 2 * b));
  odd = __any_sync(0xffffffffu, odd);
#pragma unroll
  for (int i0 = 0; i0 < WARP_KEYS / 16; i0 += KT) {
    float x[KT][NT][4];
    const uint32_t kt = i0 * 16;
    kw.template scores_q4<KT>(ks + kt * (HD / 2), kss + kt * (HD / 16), qs, sums, x);
    if (masked) {
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t bits = rows.visible(false, base, 8 * n + 2 * kw.t + h, gk) >> (2 * i0);
#pragma unroll
          for (int i = 0; i < 2 * KT; i++)
            if (!(bits >> i & 1)) x[i >> 1][n][2 * (i & 1) + h] = -INFINITY;
        }
    }
    kw.template weights<KT>(scale * KeyWarp<HD, NT, true>::CODE_UNIT, x);
#pragma unroll
    for (int i = 0; i < KT; i++) {
      const uint32_t vt = vs + (kt + 16 * i) * (HD / 2), st = vss + (kt + 16 * i) * (HD / 16);
      if (odd)
        kw.values_slow(x[i], [&](int r, int d) {
          const int b = d >> 5, j = d & 31;
          const uint32_t w = kw_lds32(vt + r * (HD / 2) + ((b ^ q4_swz<HD>(r)) << 4) + (j & 12));
          const int u = (w >> (8 * (j & 3) + (j >> 4) * 4)) & 15;
          return q4_value(u, kw_half(kw_lds16(st + r * (HD / 16) + 2 * b), 0));
        });
      else
        kw.values_q4(vt, st, x[i]);
    }
  }
}

// Sixteen of the tree's own nodes, from `node0` on: fp16 rows at ks and vs.
template <int HD, int NT>
__device__ __forceinline__ void step_nodes(KeyWarp<HD, NT, true>& kw, const UnitRows<HD, NT>& rows, uint32_t ks,
                                           uint32_t vs, uint32_t qs, float scale, int node0) {
  const int lane = threadIdx.x & 31, gk = kw.g;
  float x[1][NT][4];
  kw.scores_f16(ks, qs, x[0]);
#pragma unroll
  for (int n = 0; n < NT; n++)
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t bits = rows.visible(true, node0, 8 * n + 2 * kw.t + h, gk);
#pragma unroll
      for (int i = 0; i < 2; i++)
        if (!(bits >> i & 1)) x[0][n][2 * i + h] = -INFINITY;
    }
  kw.template weights<1>(scale, x);
  bool odd = false;
#pragma unroll
  for (int e = lane; e < 16 * (HD / 8); e += 32) {
    const uint4 v = kw_lds128(vs + e * 16);
    odd |= odd_pair(v.x) || odd_pair(v.y) || odd_pair(v.z) || odd_pair(v.w);
  }
  if (__any_sync(0xffffffffu, odd))
    kw.values_slow(x[0], [&](int r, int d) { return kw_half(kw_lds16(vs + f16_off<HD>(r, d >> 3) + 2 * (d & 7)), 0); });
  else
    kw.values_f16(vs, x[0]);
}

// Sixteen rows of k_new and v_new from node0 on to fp16 tiles; zeros from node m on.
template <int HD>
__device__ __forceinline__ void load_nodes(const TreeArgs& a, int s, int kvh, int m, int node0, uint32_t kn0, uint32_t vn0) {
  constexpr int UNITS = HD / 8;
  const int64_t from = (int64_t)s * a.nt * a.kv_stride + kvh * HD;
#pragma unroll
  for (int e = threadIdx.x & 31; e < 16 * UNITS; e += 32) {
    const int r = node0 + e / UNITS, u = e % UNITS;
    const bool ok = r < m;
    const int64_t at = from + (ok ? r : 0) * a.kv_stride + u * 8;
    kw_copy<16>(kn0 + f16_off<HD>(r, u), a.k_new + at, ok);
    kw_copy<16>(vn0 + f16_off<HD>(r, u), a.v_new + at, ok);
  }
}

// The cache row of a position of a slot, ~0 for none (2^32 rows of 64 dimensions would be 300 GB).
__device__ __forceinline__ uint32_t row_of(const TreeArgs& a, int slot, int len, int kvh, int pos) {
  if (pos >= len) return ~0u;
  const int e = a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
  const int pg = a.table[(int64_t)slot * a.max_pages + e];
  if (pg < 0 || pg >= a.n_pages) return ~0u;
  return ((uint32_t)pg * a.nkv + kvh) * a.page_size + (uint32_t)(pos - e * a.page_size);
}

template <int HD, int NT>
__global__ void __launch_bounds__(QA_THREADS, QShape<HD, NT>::RESIDENT) q4_attn_kernel(const TreeArgs a) {
  using Sh = QShape<HD, NT>;
  using KW = KeyWarp<HD, NT, true>;
  constexpr int ROWS = Sh::ROWS, STAGES = Sh::STAGES, UNITS = HD / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ TreeSmem s_tree;
  __shared__ long long s_part[QA_WARPS];
  __shared__ Start s_at;
  // (nothing behind starts early: it would take room here, 12.8 us for one node over
  // 8191 positions instead of 12.0)
  grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_cta = gridDim.x - 1;
  if ((int)blockIdx.x == n_cta) {
    plan_sequences<QA_THREADS>(a, ROWS, QA_SHIFT, n_cta, s_part, smem);
    return;
  }
  Start start;
  long long left = find_range<QA_THREADS>(a, ROWS, QA_SHIFT, n_cta, s_part, smem, &s_at, start);
  if (left <= 0) {
    check_others<QA_THREADS>(a, ROWS, QA_SHIFT, n_cta, QA_WARPS);
    return;
  }
  int s = start.s;
  long long off = start.off;
  SeqInfo q = start.q;
  bool first = true, new_tree = true;

  const uint32_t sm0 = kw_smem(smem), ring = sm0 + warp * Sh::RING;
  const uint32_t kn0 = sm0 + Sh::TREE_OFF, vn0 = kn0 + Sh::NODES * HD * 2;
  const uint32_t qs = sm0 + Sh::Q_OFF, sums = sm0 + Sh::SUM_OFF;
  const float scale = fabsf(a.scale_log2);
  const bool runs = a.page_size % WARP_KEYS == 0;
  KW kw;
  while (left > 0) {
    if (off >= q.work()) {  // the next sequence with work
      s++;
      off = 0;
      q = seq_info(a, s, ROWS, QA_SHIFT);
      new_tree = true;
      continue;
    }
    const int unit = (int)div_ll(off, q.tiles), t0 = (int)(off - (long long)unit * q.tiles);
    const int t1 = (int)min((long long)q.tiles, t0 + left);
    const int kvh = unit % a.nkv, row0 = unit / a.nkv * ROWS, M = q.m * a.G;
    const int n_sink = q.n_sink, w_tile = q.w_tile, last = q.tiles - 1;
    auto tile_base = [&](int t) { return (t < n_sink ? t : w_tile + t - n_sink) * QA_KEYS; };
    // the cache row of this lane's position of tile t: looked up a tile ahead of its load
    auto lookup = [&](int t) {
      return t < t1 && t != last ? row_of(a, q.slot, q.len, kvh, tile_base(t) + warp * WARP_KEYS + lane) : ~0u;
    };
    auto load_tile = [&](int t, uint32_t at) {
      if (t != last) {
        load_codes<HD>(ring + (t % STAGES) * Sh::STAGE, at, runs, a.k_qs, a.v_qs, a.k_scales, a.v_scales);
      } else if (16 * warp < q.m) {  // this warp's sixteen nodes
        load_nodes<HD>(a, s, kvh, q.m, 16 * warp, kn0, vn0);
      }
    };

    // ---- the piece's first tiles, and its q rows
    uint32_t ahead[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; i++) ahead[i] = lookup(t0 + i);
    if (new_tree) load_tree(a, s, q.m, s_tree);
    new_tree = false;
    __syncthreads();  // the last piece's exchange and q rows have been read
#pragma unroll
    for (int i = 0; i < STAGES - 1; i++) {
      if (t0 + i < t1) load_tile(t0 + i, ahead[i]);
      asm volatile("cp.async.commit_group;");
    }
    KW::put_queries(qs, sums, tid, QA_THREADS, a.scale_log2 < 0.0f, [&](int r) -> const __half* {
      const int m = row0 + r;
      if (m >= M) return nullptr;
      const int node = node_of(a, m);
      return a.q + ((int64_t)s * a.nt + node) * a.q_stride + (kvh * a.G + m - node * a.G) * HD;
    });
    __syncthreads();
    kw.begin();
    const UnitRows<HD, NT> rows = {a, s_tree, q.len, row0, M};

    for (int t = t0; t < t1; t++) {
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
      __syncwarp();
      if (t + STAGES - 1 < t1) load_tile(t + STAGES - 1, ahead[STAGES - 1]);
      asm volatile("cp.async.commit_group;");
      ahead[STAGES - 1] = lookup(t + STAGES);
      if (t == last) {
        if (16 * warp >= q.m) continue;
        step_nodes(kw, rows, kn0 + f16_off<HD>(16 * warp, 0), vn0 + f16_off<HD>(16 * warp, 0), qs, scale, 16 * warp);
        continue;
      }
      const int base = tile_base(t) + warp * WARP_KEYS;
      const bool masked = base + WARP_KEYS > q.len ||
                          (a.window > 0 && base + WARP_KEYS > q.sinks && base < q.lo + SPEC_MAX_TREE);
      step_codes(kw, rows, ring + (t % STAGES) * Sh::STAGE, qs, sums, scale, base, masked);
    }
    // ---- the end of the piece: the warps' results through shared memory
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the rings have been read
    float* x = reinterpret_cast<float*>(smem);
    float2(*s_ml)[ROWS] = reinterpret_cast<float2(*)[ROWS]>(x + (size_t)QA_WARPS * ROWS * Sh::XROW);
    kw.template put<Sh::XROW>(x + (size_t)warp * ROWS * Sh::XROW, s_ml[warp]);
    __syncthreads();
    const bool whole = t0 == 0 && t1 == q.tiles;
    const size_t slot = (size_t)blockIdx.x * 2 + (first ? 0 : 1);
#pragma unroll
    for (int e0 = 0; e0 < ROWS * UNITS; e0 += QA_THREADS) {
      const int e = e0 + tid;
      if (ROWS * UNITS % QA_THREADS != 0 && e >= ROWS * UNITS) break;
      // rows of the output are contiguous, rows of a piece are neighbours
      const int r = whole ? e / UNITS : e % ROWS, u = whole ? e % UNITS : e / ROWS, m = row0 + r;
      if (m >= M) continue;
      float m2 = -INFINITY;
#pragma unroll
      for (int k = 0; k < QA_WARPS; k++) m2 = fmaxf(m2, s_ml[k][r].x);
      const float ref = m2 == -INFINITY ? 0.0f : m2;
      float acc[8] = {}, l = 0.0f;
#pragma unroll
      for (int k = 0; k < QA_WARPS; k++) {
        const float2 ml = s_ml[k][r];
        const float wk = kw_exp2(ml.x - ref);
        l = fmaf(ml.y, wk, l);
        const float4* src = reinterpret_cast<const float4*>(x + ((size_t)k * ROWS + r) * Sh::XROW + u * 8);
        const float4 s0 = src[0], s1 = src[1];
        const float v[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int d = 0; d < 8; d++) acc[d] = fmaf(v[d], wk, acc[d]);
      }
      if (whole) {
        const float inv = 1.0f / l;
        const int node = node_of(a, m), hd = kvh * a.G + m - node * a.G;
        *reinterpret_cast<uint4*>(a.out + (((int64_t)s * a.nt + node) * a.nq + hd) * HD + u * 8) =
            make_uint4(kw_pack(acc[0] * inv, acc[1] * inv), kw_pack(acc[2] * inv, acc[3] * inv),
                       kw_pack(acc[4] * inv, acc[5] * inv), kw_pack(acc[6] * inv, acc[7] * inv));
      } else {
        float4* po = reinterpret_cast<float4*>(a.part_o) + (slot * (HD / 4) + 2 * u) * ROWS + r;
        po[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        po[ROWS] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (u == 0) a.part_ml[slot * ROWS + r] = make_float2(m2, l);
      }
    }
    left -= t1 - t0;
    off += t1 - t0;
    first = false;
  }
  check_others<QA_THREADS>(a, ROWS, QA_SHIFT, n_cta, QA_WARPS);
}

// ---------------------------------------------------------------------------
// Small calls, and short sequences: a cluster of CTAs has a unit (sequence, kv head), its
// positions are dealt to their warps 32 at a time, and the results are joined through distributed shared
// memory: no cut to be found, no second kernel.
// ---------------------------------------------------------------------------
constexpr int QU_WARPS = 8, QU_THREADS = 32 * QU_WARPS;

template <int HD, int NT>
struct UShape : QShape<HD, NT> {
  using Q = QShape<HD, NT>;
  using Join = JoinShape<HD, Q::ROWS, QU_WARPS>;
  static constexpr int TREE_OFF = ((QU_WARPS * Q::RING > Join::EXCHANGE ? QU_WARPS * Q::RING : Join::EXCHANGE) + 127) / 128 * 128;
  static constexpr int Q_OFF = TREE_OFF + 2 * Q::NODES * HD * 2;
  static constexpr int SUM_OFF = Q_OFF + KeyWarp<HD, NT, true>::Q_BYTES;
  static constexpr int PART_OFF = (SUM_OFF + KeyWarp<HD, NT, true>::SUM_BYTES + 127) / 128 * 128;
  static constexpr size_t SMEM = PART_OFF + Join::PART;
  static constexpr int RESIDENT = NT == 4 ? 1 : HD == 64 ? 3 : NT == 2 ? 1 : 2;
};

struct UnitArgs {
  TreeArgs t;
  int ranks;
};

template <int HD, int NT>
__global__ void __launch_bounds__(QU_THREADS, UShape<HD, NT>::RESIDENT) q4_unit_kernel(const UnitArgs u) {
  using Sh = UShape<HD, NT>;
  using KW = KeyWarp<HD, NT, true>;
  constexpr int ROWS = Sh::ROWS, STAGES = Sh::STAGES, UNITS = HD / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ TreeSmem s_tree;
  // (the same, called in a row: a window of 4096 for 16 sequences 11.5 us instead of 11.7 to 14;
  // in a graph 11.2 instead of 10.9)
  grid_dep_wait();
  const TreeArgs& a = u.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % u.ranks, unit = blockIdx.x / u.ranks, kvh = unit % a.nkv, s = unit / a.nkv;
  const SeqInfo q = seq_info(a, s, ROWS, QA_SHIFT);
  const uint32_t sm0 = kw_smem(smem), ring = sm0 + warp * Sh::RING;
  const uint32_t kn0 = sm0 + Sh::TREE_OFF, vn0 = kn0 + Sh::NODES * HD * 2;
  const uint32_t qs = sm0 + Sh::Q_OFF, sums = sm0 + Sh::SUM_OFF;
  // steps of 32 positions: of the sinks, then from the window's first on
  const int sink_steps = (q.sinks + WARP_KEYS - 1) / WARP_KEYS;
  const int from = max(q.lo / WARP_KEYS, sink_steps);
  const int steps = sink_steps + max(0, (q.len + WARP_KEYS - 1) / WARP_KEYS - from);
  auto step_base = [&](int i) { return (i < sink_steps ? i : from + i - sink_steps) * WARP_KEYS; };
  const int warps = u.ranks * QU_WARPS, gw = rank * QU_WARPS + warp;
  const int nodes0 = 16 * (warps - 1 - gw);  // the tree's nodes of this warp: the last warps have few steps
  const bool has_nodes = warps - 1 - gw < 2 && nodes0 < q.m;
  const bool runs = a.page_size % WARP_KEYS == 0;
  auto lookup = [&](int i) { return i < steps ? row_of(a, q.slot, q.len, kvh, step_base(i) + lane) : ~0u; };
  auto load = [&](int stage, uint32_t at) {
    load_codes<HD>(ring + stage * Sh::STAGE, at, runs, a.k_qs, a.v_qs, a.k_scales, a.v_scales);
  };
  uint32_t ahead = lookup(gw);
  if (has_nodes) load_nodes<HD>(a, s, kvh, q.m, nodes0, kn0, vn0);
  if (gw < steps) load(0, ahead);
  asm volatile("cp.async.commit_group;");
  ahead = lookup(gw + warps);
  // the sequence's status: slot, length and count, pages that somebody sees, tree
  int st = q.bad;
  if (q.bad == 0) {
    bool bad = false;
    const int held = q.m == 0 || q.len == 0 ? 0 : (q.len - 1) / a.page_size + 1;
    const int e1 = q.sinks > 0 ? min(held, (q.sinks - 1) / a.page_size + 1) : 0;
    const int e0 = max(q.lo < q.len ? q.lo / a.page_size : held, e1);
    const int32_t* row = a.table + (int64_t)q.slot * a.max_pages;
    for (int e = tid; e < e1 + max(0, held - e0); e += QU_THREADS) {
      const int p = row[e < e1 ? e : e0 + e - e1];
      bad |= p < 0 || p >= a.n_pages;
    }
    if (!load_tree(a, s, q.m, s_tree)) st |= SPEC_ST_TREE;
    if (__syncthreads_or(bad)) st |= SPEC_ST_PAGE;
  }
  if (kvh == 0 && rank == 0 && tid == 0) a.status[s] = st;
  const int M = q.m * a.G;
  if (st != 0 || q.m == 0) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (st == 0 || rank != 0) return;
    const int m = a.n_nodes != nullptr ? a.n_nodes[s] : a.nt, nodes = m < 0 || m > a.nt ? a.nt : m;
    for (int e = tid; e < nodes * a.G * UNITS; e += QU_THREADS) {
      const int r = e / UNITS, node = node_of(a, r);
      *reinterpret_cast<uint4*>(a.out + (((int64_t)s * a.nt + node) * a.nq + kvh * a.G + r - node * a.G) * HD +
                                e % UNITS * 8) = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
    }
    return;
  }
  KW::put_queries(qs, sums, tid, QU_THREADS, a.scale_log2 < 0.0f, [&](int r) -> const __half* {
    if (r >= M) return nullptr;
    const int node = node_of(a, r);
    return a.q + ((int64_t)s * a.nt + node) * a.q_stride + (kvh * a.G + r - node * a.G) * HD;
  });
  __syncthreads();
  const float scale = fabsf(a.scale_log2);
  const UnitRows<HD, NT> rows = {a, s_tree, q.len, 0, M};
  KW kw;
  kw.begin();
  int stage = 0;
  for (int i = gw; i < steps; i += warps) {
    __syncwarp();  // the last stage has been read
    if (i + warps < steps) load(stage ^ 1, ahead);
    asm volatile("cp.async.commit_group;");
    ahead = lookup(i + 2 * warps);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    const int base = step_base(i);
    const bool masked = base + WARP_KEYS > q.len ||
                        (a.window > 0 && base + WARP_KEYS > q.sinks && base < q.lo + SPEC_MAX_TREE);
    step_codes(kw, rows, ring + stage * Sh::STAGE, qs, sums, scale, base, masked);
    stage ^= 1;
  }
  static_assert(STAGES == 2, "a stage in use, a stage on its way");
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  if (has_nodes)
    step_nodes(kw, rows, kn0 + f16_off<HD>(nodes0, 0), vn0 + f16_off<HD>(nodes0, 0), qs, scale, nodes0);
  __syncthreads();  // the rings have been read
  join_unit<QU_WARPS>(kw, smem, Sh::PART_OFF, rank, u.ranks, M, [&](int r, int x, const float (&acc)[8], float l) {
    const int node = node_of(a, r);
    put_row(a.out + (((int64_t)s * a.nt + node) * a.nq + kvh * a.G + r - node * a.G) * HD + x * 8, acc, l);
  });
}

// Query rows of a unit.  Up to 32 rows run here, more on the tcgen05 kernel with 64,
// 128 or 256 that share one read of the cache (tree_attn_tc.cu).  With 32 rows that one takes
// 20.1 us where this takes 16.6 (16 sequences of 500 positions), 36.5 and 35.5 (4 of
// 8000), 181 and 198 (4 of 65536; no length is known here), with 16 rows 184 and 108.
int q4_rows(int M) { return M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256; }
bool q4_on_tc(int rows) { return rows >= 64; }

int q4_resident(int hd, int rows) {
  return q4_on_tc(rows) ? 1
         : rows == 32   ? QShape<128, 4>::RESIDENT
         : hd == 64     ? (rows == 16 ? QShape<64, 2>::RESIDENT : QShape<64, 1>::RESIDENT)
         : rows == 16   ? QShape<128, 2>::RESIDENT
                        : QShape<128, 1>::RESIDENT;
}
// The CTAs with tiles: what is resident, but for the one that plans.
int q4_ctas(int hd, int rows) { return std::max(1, q4_resident(hd, rows) * device_sms() - 1); }

template <int HD, int NT>
cudaError_t launch_q4(const TreeArgs& a, int n_cta, cudaStream_t st) {
  return launch_dependent(q4_attn_kernel<HD, NT>, n_cta + 1, QA_THREADS, QShape<HD, NT>::SMEM, st, a);
}
template <int HD>
cudaError_t launch_q4_rows(const TreeArgs& a, int n_cta, cudaStream_t st) {
  return a.rows == 8    ? launch_q4<HD, 1>(a, n_cta, st)
         : a.rows == 16 ? launch_q4<HD, 2>(a, n_cta, st)
                        : launch_q4<HD, 4>(a, n_cta, st);
}
// CTAs of a unit in the clusters' form, or 0 for the cut's: up to eight (clusters of more
// leave SMs of a GPC unused), one an SM, as long as each warp has a step of 32 positions.  The
// lengths are on the device; what counts here is the most positions that a sequence can
// have: its table's, or the window's.  Clusters take
//   up to three steps a warp anywhere (one sequence of 1000 positions 8.2 us against the cut's
//   10.0; of 16000, eight steps on 64 SMs, 16.7 and 14.1: not there);
//   up to eight where the CTAs are three quarters of the SMs, and with up to 8 rows up to sixteen;
//   of more than two units an SM those with up to 8 rows (160 of 300, 14 heads over 2 of 64, 8.0
//   against 17; 16 rows, 100 of 1000, 76 and 66: not there).
// With tables of 4096 positions and up to 8 rows 20 to 28, 39 to 56 and 77 to 113 units so go
// to the cut, all others to clusters.  These and the cut there, 8 kv heads of 128, n sequences of
// 4000: n = 4 12.5 and 18.0, 8 17.7 and 26.5, 16 27 and 32, 20 40 and 38, 32 42 and 53, 40 62
// and 59, 64 79 and 82; of 1000 in such tables 16 11.6 and 17.0, 64 29 and 30.  What this
// costs are batches of one long sequence among short ones, of which the cut gives all CTAs a
// part: 4000 beside 100 for each of the others n = 16 25.6 and 15.5, 36 26 and 16.5, 64 27 and 23;
// lengths spread evenly up to 4000 n = 16 25 and 20, 36 33 and 39, 64 51 and 58.  Between the
// ranges two CTAs a unit would be faster for 5 to 9 sequences (5 of 4000 21.4 us by the cut, 17.4 so;
// 10 22 and 24).
int unit_ranks(const TreeArgs& a) {
  const int64_t units = (int64_t)a.n_seq * a.nkv, all = (int64_t)a.max_pages * a.page_size;
  const int64_t most = a.window > 0 ? std::min<int64_t>(all, (int64_t)a.window + a.sinks + 2 * WARP_KEYS) : all;
  const int64_t steps = (most + WARP_KEYS - 1) / WARP_KEYS, sms = device_sms();
  const int most_steps = a.rows == 8 ? 16 : 8;
  if (units > 2 * sms) return a.rows == 8 && steps <= (int64_t)QU_WARPS * most_steps ? 1 : 0;
  int ranks = 1;
  while (ranks < 8 && units * ranks * 2 <= sms && steps >= (int64_t)QU_WARPS * ranks * 2) ranks *= 2;
  return steps <= (int64_t)QU_WARPS * ranks * (4 * units * ranks >= 3 * sms ? most_steps : 3) ? ranks : 0;
}

template <int HD, int NT>
cudaError_t launch_unit(const TreeArgs& a, int ranks, cudaStream_t st) {
  const UnitArgs u = {a, ranks};
  return launch_clusters(q4_unit_kernel<HD, NT>, u, (size_t)a.n_seq * a.nkv * ranks, QU_THREADS, ranks,
                         UShape<HD, NT>::SMEM, st);
}
template <int HD>
cudaError_t launch_unit_rows(const TreeArgs& a, int ranks, cudaStream_t st) {
  return a.rows == 8    ? launch_unit<HD, 1>(a, ranks, st)
         : a.rows == 16 ? launch_unit<HD, 2>(a, ranks, st)
                        : launch_unit<HD, 4>(a, ranks, st);
}

template <int HD, int NT>
void init_q4() {
  cudaFuncSetAttribute(q4_attn_kernel<HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)QShape<HD, NT>::SMEM);
  cudaFuncSetAttribute(q4_unit_kernel<HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)UShape<HD, NT>::SMEM);
}

}  // namespace

void q4_init_attrs() {
  init_q4<64, 1>();
  init_q4<64, 2>();
  init_q4<64, 4>();
  init_q4<128, 1>();
  init_q4<128, 2>();
  init_q4<128, 4>();
}

int q4_workspace(const spec_pages_q4* kv, int n_seq, int nt, int n_q_heads, size_t* bytes) {
  const int rc = check_pages_q4(kv, true);
  if (rc != SPEC_OK) return rc;
  const spec_pages book = book_of(kv);
  const int rc2 = tree_check(&book, n_seq, nt, n_q_heads);
  if (rc2 != SPEC_OK) return rc2;
  const int rows = q4_rows(nt * (n_q_heads / kv->n_kv_heads));
  *bytes = tree_scratch(kv->head_dim, rows, q4_ctas(kv->head_dim, rows), n_seq);
  return SPEC_OK;
}

int launch_tree_q4(const spec_pages_q4* kv, int layer, const spec_tree* t, const uint16_t* q, int64_t q_stride,
                   const uint16_t* k_new, const uint16_t* v_new, int64_t kv_stride, uint16_t* out, void* workspace,
                   int32_t* status, cudaStream_t st) {
  TreeArgs a;
  const spec_pages book = book_of(kv);
  const int hd = kv->head_dim, rows = q4_rows(t->nt * (t->n_q_heads / kv->n_kv_heads)), n_cta = q4_ctas(hd, rows);
  tree_fill(a, &book, 0, t, q, q_stride, k_new, v_new, kv_stride, out, workspace, status, rows,
            q4_on_tc(rows) ? TREE_TC_SHIFT : QA_SHIFT, n_cta, q4_on_tc(rows));
  const int64_t row = (int64_t)layer * kv->layer_stride;
  a.k_qs = kv->k_qs + row * (hd / 2);
  a.v_qs = kv->v_qs + row * (hd / 2);
  a.k_scales = reinterpret_cast<const __half*>(kv->k_scales) + row * (hd / 32);
  a.v_scales = reinterpret_cast<const __half*>(kv->v_scales) + row * (hd / 32);
  const int ranks = q4_on_tc(rows) ? 0 : unit_ranks(a);
  if (ranks > 0) {
    const cudaError_t e = hd == 128 ? launch_unit_rows<128>(a, ranks, st) : launch_unit_rows<64>(a, ranks, st);
    return e == cudaSuccess ? SPEC_OK
                            : fail(SPEC_E_CUDA, std::string("4-bit tree attention: ") + cudaGetErrorString(e));
  }
  cudaError_t e = q4_on_tc(rows) ? tree_tc_launch(a, hd, n_cta, st)
                  : hd == 128    ? launch_q4_rows<128>(a, n_cta, st)
                                 : launch_q4_rows<64>(a, n_cta, st);
  if (e == cudaSuccess) e = tree_join_launch(a, hd, n_cta, st);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("4-bit tree attention: ") + cudaGetErrorString(e));
  return SPEC_OK;
}
