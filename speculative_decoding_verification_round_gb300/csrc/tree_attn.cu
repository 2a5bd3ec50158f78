// tree_attn.cu -- attention of drafted trees over a paged cache, with an
// optional sliding window and sink positions (spec_tree_attn).
//
// Every query row of one (sequence, kv head) -- nodes x GQA group -- reads the
// same keys, so the rows are the M of an MMA tile and the cache is streamed
// once for all of them: S = Q K^T, a softmax with a running maximum and sum in
// fp32 (log2 domain), O = P V, over tiles of 64 positions.  The tree's own
// nodes are the last tile, masked by each node's set of ancestors.  The kernel
// here has 16 or 32 rows; more go to tree_attn_tc.cu.
//
// Work is cut evenly whatever the lengths are: the (sequence, kv head, row
// block) units, each of its own number of tiles, are laid end to end, and every
// CTA takes as many tiles of them.  The lengths are only known on the device,
// so every CTA derives the cut from them.  A unit that one CTA holds whole is
// written by it; the pieces of a cut unit (at most two a CTA) go to the
// workspace as (max, sum, unnormalised O) and a second kernel joins them in the
// order of the positions.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "tree_attn.cuh"

namespace {

constexpr int TT_SHIFT = 6, TT_KEYS = 1 << TT_SHIFT;  // positions per tile
constexpr int TT_THREADS = 128;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// Two floats as packed fp16, the first in the low half; and back.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  float2 f;
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
      : "=f"(f.x), "=f"(f.y) : "r"(v));
  return f;
}
// 2^x (0 below the normal range, which no sum here can tell apart).
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 16 bytes to shared memory; zeros if !valid (src is then any readable address).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0));
}
// Byte offset of 16-byte unit u of row r in a swizzled tile.
template <int HD>
__device__ __forceinline__ uint32_t tile_off(int r, int u) {
  return (uint32_t)(r * (HD * 2) + ((u ^ (r & 7)) << 4));
}

// ---------------------------------------------------------------------------
// the main kernel.  Each of four warps has all rows (MT m16 tiles) against 16
// keys of every tile, with its own running (max, sum, O), joined at the end of
// a piece: few rows have to share the keys among the warps.
//
// 2 x rows flops per byte of K (twice that for P V, whose weights are a pair)
// keep mma.sync within the memory's time up to 32 rows.  Long contexts are
// bound by the memory: 64 sequences of 32768 positions, one node each, 14
// query heads over 2 of 64 dimensions (1.0 GB), take 170 us, 5.9 TB/s, 87% of
// the copy bandwidth.  Short ones are bound by their chain of latencies: 8
// nodes over 4096 positions, 32 heads over 8 of 128 (17 MB) 15 us, of which 2
// the cut, 2.5 the tree, the page lookups and the first loads, 4 two tiles, 2
// the piece's end and 3 the joining kernel.
// ---------------------------------------------------------------------------
// CTAs of an SM: two of 128 dimensions (three with two stages each: no gain,
// 64 sequences of one node over 512 positions 74 -> 78 us), four of 64
// dimensions and 16 rows (16 sequences of 32768 positions 56 us with three, 54
// with four; with a window of 4096 17.2 us with two, 15.6 with four).
constexpr int resident(int hd, int rows) { return hd == 64 && rows == 16 ? 4 : 2; }

// Factor of weights and sums: a weight w, at most 1, goes to the MMA as a pair
// of fp16 numbers, which holds all of it but 2^-20 w + 2^-39 with the factor and
// all but 2^-20 w + 2^-24 without (16 nats below a row's largest, 6% off).
constexpr float P_FACTOR = 32768.0f;

template <int HD, int MT>
struct Shape {
  static constexpr int ROWS = 16 * MT;
  static constexpr int RESIDENT = resident(HD, ROWS), STAGES = 3;
  static constexpr int KG = TT_THREADS / 32;
  static constexpr int KEYS = TT_KEYS / KG;
  static constexpr int TILE = TT_KEYS * HD * 2;  // bytes of a K (or V) tile
  static constexpr int XROW = HD + 8;            // floats of an exchange row (padded)
  static constexpr size_t Q_OFF = (size_t)STAGES * 2 * TILE;
  static constexpr size_t SMEM = Q_OFF + (size_t)ROWS * HD * 2;
  static_assert((size_t)KG * ROWS * (XROW * 4 + 8) <= Q_OFF, "the exchange fits over the tiles");
};

template <int HD, int MT>
__global__ void __launch_bounds__(TT_THREADS, Shape<HD, MT>::RESIDENT) tree_attn_kernel(const TreeArgs a) {
  using Sh = Shape<HD, MT>;
  constexpr int ROWS = Sh::ROWS, STAGES = Sh::STAGES, KG = Sh::KG, KEYS = Sh::KEYS, NB = KEYS / 8, UNITS = HD / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ TreeSmem s_tree;
  __shared__ long long s_part[TT_THREADS / 32];
  __shared__ Start s_at;
  grid_dep_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int kg = warp;  // this warp's key group

  const int n_cta = gridDim.x - 1;
  if ((int)blockIdx.x == n_cta) {
    plan_sequences<TT_THREADS>(a, ROWS, TT_SHIFT, n_cta, s_part, smem);
    return;
  }
  Start start;
  long long left = find_range<TT_THREADS>(a, ROWS, TT_SHIFT, n_cta, s_part, smem, &s_at, start);
  if (left <= 0) {
    check_others<TT_THREADS>(a, ROWS, TT_SHIFT, n_cta, TT_THREADS / 32);
    return;
  }
  int s = start.s;
  long long off = start.off;
  SeqInfo q = start.q;
  bool first = true, new_tree = true;  // piece of this CTA; of its sequence

  const uint32_t sm0 = smem_u32(smem), qs0 = sm0 + (uint32_t)Sh::Q_OFF;
  const int lu = tid % UNITS, lr = tid / UNITS;  // this thread's unit and first row of a tile
  constexpr int LR = TT_THREADS / UNITS, WR = 32 / UNITS;  // rows of a pass, and of a warp in it
  // the row of a tile that this lane looks up for its warp
  const int my_row = (lane % 16) / WR * LR + warp * WR + lane % WR;
  while (left > 0) {
    if (off >= q.work()) {  // the next sequence with work
      s++;
      off = 0;
      q = seq_info(a, s, ROWS, TT_SHIFT);
      new_tree = true;
      continue;
    }
    const int unit = (int)div_ll(off, q.tiles), t0 = (int)(off - (long long)unit * q.tiles);
    const int t1 = (int)min((long long)q.tiles, t0 + left);
    const int kvh = unit % a.nkv, row0 = unit / a.nkv * ROWS, M = q.m * a.G;

    // positions of tile t (context tiles only)
    const int n_sink = q.n_sink, w_tile = q.w_tile, last = q.tiles - 1;
    auto tile_base = [&](int t) { return (t < n_sink ? t : w_tile + t - n_sink) * TT_KEYS; };
    // The cache row (or the tree's node) of this lane's row of tile t, ~0 for
    // zeros: looked up a tile ahead of its load, as the table is memory, too.
    // (2^32 rows would be 550 GB.)
    auto lookup = [&](int t) {
      uint32_t x = ~0u;
      if (t == last) {
        if (my_row < q.m) x = (uint32_t)my_row;
      } else if (t < t1) {
        const int pos = tile_base(t) + my_row;
        if (pos < q.len) {
          const int e = a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
          const int pg = a.table[(int64_t)q.slot * a.max_pages + e];
          if (pg >= 0 && pg < a.n_pages)
            x = ((uint32_t)pg * a.nkv + kvh) * a.page_size + (uint32_t)(pos - e * a.page_size);
        }
      }
      return x;
    };
    auto load_tile = [&](int t, uint32_t at) {
      const uint32_t ks = sm0 + (uint32_t)(t % STAGES) * 2 * Sh::TILE, vs = ks + Sh::TILE;
      const bool tree = t == last;
      const int64_t row = tree ? a.kv_stride : HD, from = tree ? (int64_t)s * a.nt * a.kv_stride + kvh * HD : 0;
      const __half* kp = (tree ? a.k_new : a.k) + from + lu * 8;
      const __half* vp = (tree ? a.v_new : a.v) + from + lu * 8;
#pragma unroll
      for (int i = 0; i < TT_KEYS / LR; i++) {
        const uint32_t x = __shfl_sync(0xffffffffu, at, i * WR + lane / UNITS);
        const bool ok = x != ~0u;
        const int64_t off = (int64_t)(ok ? x : 0u) * row;
        cp16(ks + tile_off<HD>(lr + i * LR, lu), kp + off, ok);
        cp16(vs + tile_off<HD>(lr + i * LR, lu), vp + off, ok);
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
      if (i == 0) {
        for (int e = tid; e < ROWS * UNITS; e += TT_THREADS) {
          const int r = e / UNITS, u = e % UNITS, m = row0 + r;
          const bool ok = m < M;
          const int node = ok ? node_of(a, m) : 0, h = kvh * a.G + (ok ? m - node * a.G : 0);
          cp16(qs0 + tile_off<HD>(r, u), a.q + ((int64_t)s * a.nt + node) * a.q_stride + h * HD + u * 8, ok);
        }
      }
      asm volatile("cp.async.commit_group;");
    }
    // this thread's rows: [tile][upper half]
    int pos[MT][2];
    unsigned long long anc[MT][2];
    float mx[MT][2], sum[MT][2], o[MT][HD / 8][4];
#pragma unroll
    for (int i = 0; i < MT; i++) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int m = row0 + i * 16 + h * 8 + g;
        const int node = m < M ? node_of(a, m) : 0;
        pos[i][h] = q.len + s_tree.depth[node];
        anc[i][h] = m < M ? s_tree.anc[node] : 0ull;
        mx[i][h] = -INFINITY;
        sum[i][h] = 0.0f;
      }
#pragma unroll
      for (int d = 0; d < HD / 8; d++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[i][d][e] = 0.0f;
    }
    const int q_row = (lane & 7) + ((lane >> 3) & 1) * 8;  // ldmatrix row of a q fragment

    for (int t = t0; t < t1; t++) {
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
      __syncthreads();
      if (t + STAGES - 1 < t1) load_tile(t + STAGES - 1, ahead[STAGES - 1]);
      asm volatile("cp.async.commit_group;");
      ahead[STAGES - 1] = lookup(t + STAGES);
      const uint32_t ks = sm0 + (uint32_t)(t % STAGES) * 2 * Sh::TILE, vs = ks + Sh::TILE;
      const int key0 = kg * KEYS;

      // ---- S = Q K^T
      float sc[MT][NB][4];
#pragma unroll
      for (int i = 0; i < MT; i++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
          for (int e = 0; e < 4; e++) sc[i][nb][e] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < HD / 16; kk += 2) {
        uint32_t qa[MT][2][4];
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
          for (int j = 0; j < 2; j++)
            ldsm_x4(qs0 + tile_off<HD>(i * 16 + q_row, 2 * (kk + j) + (lane >> 4)), qa[i][j]);
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
          uint32_t b[4];
          ldsm_x4(ks + tile_off<HD>(key0 + 8 * nb + (lane & 7), 2 * kk + (lane >> 3)), b);
#pragma unroll
          for (int i = 0; i < MT; i++) {
            mma_16816(sc[i][nb], qa[i][0], b[0], b[1]);
            mma_16816(sc[i][nb], qa[i][1], b[2], b[3]);
          }
        }
      }
      // ---- scale and mask
      const int base = t == last ? 0 : tile_base(t);
      const bool masked = t == last || base + TT_KEYS > q.len ||
                          (a.window > 0 && base + TT_KEYS > q.sinks && base < q.lo + SPEC_MAX_TREE);
#pragma unroll
      for (int i = 0; i < MT; i++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            float x = sc[i][nb][e] * a.scale_log2;
            if (masked) {
              const int h = e >> 1, key = key0 + 8 * nb + 2 * t4 + (e & 1);
              bool see;
              int p;
              if (t == last) {
                see = (anc[i][h] >> key) & 1;
                p = q.len + (see ? s_tree.depth[key] : 0);
              } else {
                p = base + key;
                see = p < q.len;
              }
              if (a.window > 0) see = see && (p < a.sinks || p > pos[i][h] - a.window);
              x = see ? x : -INFINITY;
            }
            sc[i][nb][e] = x;
          }
      // ---- running maximum and sum
#pragma unroll
      for (int i = 0; i < MT; i++) {
        float nm[2], al[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float m2 = mx[i][h];
#pragma unroll
          for (int nb = 0; nb < NB; nb++) m2 = fmaxf(m2, fmaxf(sc[i][nb][2 * h], sc[i][nb][2 * h + 1]));
          m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
          m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
          nm[h] = m2 == -INFINITY ? 0.0f : m2;  // a row without a visible key so far
          al[h] = exp2_fast(mx[i][h] - nm[h]);
          mx[i][h] = m2;
          float l = 0.0f;
#pragma unroll
          for (int nb = 0; nb < NB; nb++) {
            sc[i][nb][2 * h] = exp2_fast(sc[i][nb][2 * h] - nm[h]) * P_FACTOR;
            sc[i][nb][2 * h + 1] = exp2_fast(sc[i][nb][2 * h + 1] - nm[h]) * P_FACTOR;
            l += sc[i][nb][2 * h] + sc[i][nb][2 * h + 1];
          }
          sum[i][h] = fmaf(sum[i][h], al[h], l);  // this lane's share of the row
        }
        if (__any_sync(0xffffffffu, al[0] != 1.0f || al[1] != 1.0f)) {
#pragma unroll
          for (int d = 0; d < HD / 8; d++) {
            o[i][d][0] *= al[0];
            o[i][d][1] *= al[0];
            o[i][d][2] *= al[1];
            o[i][d][3] *= al[1];
          }
        }
      }
      // ---- a masked tile's V may hold infinities or NaN that some rows do
      // ---- not see, and 0 * inf is NaN: such rows of V are added by the
      // ---- lanes that see them and zeroed for the MMA
      if (masked) {
        bool odd = false;
        for (int e = tid; e < TT_KEYS * UNITS; e += TT_THREADS) {
          uint32_t v[4];
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(vs + e * 16));
#pragma unroll
          for (int x = 0; x < 4; x++)
            odd |= (v[x] & 0x7C00u) == 0x7C00u || (v[x] & 0x7C000000u) == 0x7C000000u;
        }
        if (__syncthreads_or(odd)) {
#pragma unroll
          for (int i = 0; i < MT; i++)
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll 1
              for (int kb = 0; kb < 8; kb++) {
                const int src = (lane & ~3) | (kb >> 1), key = key0 + 8 * nb + kb;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                  const float pa = __shfl_sync(0xffffffffu, sc[i][nb][2 * h], src);
                  const float pb = __shfl_sync(0xffffffffu, sc[i][nb][2 * h + 1], src);
                  const float p = kb & 1 ? pb : pa;
                  if (p > 0.0f) {
#pragma unroll
                    for (int d = 0; d < HD / 8; d++) {
                      uint32_t v;
                      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(vs + tile_off<HD>(key, d) + t4 * 4));
                      const float2 f = unpack_f16(v);
                      o[i][d][2 * h] = fmaf(p, f.x, o[i][d][2 * h]);
                      o[i][d][2 * h + 1] = fmaf(p, f.y, o[i][d][2 * h + 1]);
                    }
                  }
                }
              }
          __syncthreads();
          for (int e = tid; e < TT_KEYS * UNITS; e += TT_THREADS)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vs + e * 16), "r"(0));
          __syncthreads();
        }
      }
      // ---- O += P V, with P as a pair of fp16 numbers hi + lo
#pragma unroll
      for (int kk = 0; kk < KEYS / 16; kk++) {
        uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
          for (int n = 0; n < 2; n++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const float p0 = sc[i][2 * kk + n][2 * h], p1 = sc[i][2 * kk + n][2 * h + 1];
              const float c0 = __uint_as_float(__float_as_uint(p0) & P_CUT), c1 = __uint_as_float(__float_as_uint(p1) & P_CUT);
              hi[i][2 * n + h] = pack_f16(c0, c1);
              lo[i][2 * n + h] = pack_f16(fmaf(c0, -P_REST, p0), fmaf(c1, -P_REST, p1));
            }
#pragma unroll
        for (int d = 0; d < HD / 8; d += 2) {
          uint32_t b[4];
          ldsm_x4_t(vs + tile_off<HD>(key0 + 16 * kk + (lane & 7) + ((lane >> 3) & 1) * 8, d + (lane >> 4)), b);
#pragma unroll
          for (int i = 0; i < MT; i++) {
            mma_16816(o[i][d], hi[i], b[0], b[1]);
            mma_16816(o[i][d], lo[i], b[0], b[1]);
            mma_16816(o[i][d + 1], hi[i], b[2], b[3]);
            mma_16816(o[i][d + 1], lo[i], b[2], b[3]);
          }
        }
      }
    }
    // ---- the end of the piece: the key groups' results through shared
    // ---- memory, added in the order of the groups
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the tiles have been read
    float* x = reinterpret_cast<float*>(smem);
    float2(*s_ml)[16 * MT] = reinterpret_cast<float2(*)[16 * MT]>(x + (size_t)KG * ROWS * Sh::XROW);
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float l = sum[i][h];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int r = i * 16 + h * 8 + g;
        if (t4 == 0) s_ml[warp][r] = make_float2(mx[i][h], l);
        float* dst = x + ((size_t)kg * ROWS + r) * Sh::XROW + 2 * t4;
#pragma unroll
        for (int d = 0; d < HD / 8; d++)
          *reinterpret_cast<float2*>(dst + 8 * d) = make_float2(o[i][d][2 * h], o[i][d][2 * h + 1]);
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == q.tiles;
    const size_t slot = (size_t)blockIdx.x * 2 + (first ? 0 : 1);
#pragma unroll
    for (int e0 = 0; e0 < ROWS * UNITS; e0 += TT_THREADS) {
      const int e = e0 + tid;
      // rows of the output are contiguous, rows of a piece are neighbours
      const int r = whole ? e / UNITS : e % ROWS, u = whole ? e % UNITS : e / ROWS, m = row0 + r;
      if (m >= M) continue;
      float m2 = -INFINITY;
#pragma unroll
      for (int k = 0; k < KG; k++) m2 = fmaxf(m2, s_ml[k][r].x);
      const float ref = m2 == -INFINITY ? 0.0f : m2;
      float acc[8] = {}, l = 0.0f;
#pragma unroll
      for (int k = 0; k < KG; k++) {
        const float2 ml = s_ml[k][r];
        const float wk = exp2f(ml.x - ref);
        l = fmaf(ml.y, wk, l);
        const float4* src = reinterpret_cast<const float4*>(x + ((size_t)k * ROWS + r) * Sh::XROW + u * 8);
        const float4 s0 = src[0], s1 = src[1];
        const float v[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int d = 0; d < 8; d++) acc[d] = fmaf(v[d], wk, acc[d]);
      }
      if (whole) {
        const float inv = 1.0f / l;
        uint4 y;
        y.x = pack_f16(acc[0] * inv, acc[1] * inv);
        y.y = pack_f16(acc[2] * inv, acc[3] * inv);
        y.z = pack_f16(acc[4] * inv, acc[5] * inv);
        y.w = pack_f16(acc[6] * inv, acc[7] * inv);
        const int node = node_of(a, m), hd = kvh * a.G + m - node * a.G;
        *reinterpret_cast<uint4*>(a.out + (((int64_t)s * a.nt + node) * a.nq + hd) * HD + u * 8) =
            y;
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
  check_others<TT_THREADS>(a, ROWS, TT_SHIFT, n_cta, TT_THREADS / 32);
}

// ---------------------------------------------------------------------------
// the joining kernel: a CTA has 32 rows (node, head) of one kv head, a lane a
// row and 8 dimensions, eight pieces' loads in flight together.  Joins the
// pieces of the rows' unit in the order of the positions, or writes NaN for a
// sequence in error.  SPLIT: the CTA has 8 dimensions and its warps an eighth
// of the pieces each (the kernel for few rows cuts a long context into dozens
// of pieces: 8 nodes over 4096 positions, 33 pieces, 22 us without, 18 with
// four warps, 16.3 -> 15.1 with eight); otherwise every warp has all pieces of
// its dimensions (12 x 16 nodes 37 -> 29 us), the CTA 32 of them a turn, so
// that many units, most of them whole, take no more CTAs than fit at once
// (64 sequences of one node over 512 positions: 44 of 74 us were spent here
// with a CTA per 8 dimensions, now 38 in all).
// ---------------------------------------------------------------------------
constexpr int TJ_ROWS = 32;
constexpr int join_warps(bool split) { return split ? 8 : 4; }

template <int HD, bool SPLIT>
__global__ void __launch_bounds__(32 * join_warps(SPLIT))
tree_join_kernel(const TreeArgs a, int blocks, int slices) {
  constexpr int TJ_WARPS = join_warps(SPLIT), TJ_THREADS = 32 * TJ_WARPS;
  __shared__ float s_o[TJ_WARPS][8][TJ_ROWS];
  __shared__ float2 s_ml[TJ_WARPS][TJ_ROWS];
  const int slice = blockIdx.x % slices, kvh = blockIdx.x / slices % a.nkv;
  const int blk = blockIdx.x / (slices * a.nkv) % blocks, s = blockIdx.x / (slices * a.nkv) / blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int m = blk * TJ_ROWS + lane, r = m & (a.rows - 1), node = node_of(a, m);
  grid_dep_begin();
  const longlong2 p0 = __ldcg(reinterpret_cast<const longlong2*>(a.plan + s));
  const int4 p1 = __ldcg(reinterpret_cast<const int4*>(a.plan + s) + 1);
  const long long before = p0.x, share = p0.y;
  const int tiles = p1.x, padded = p1.y, nodes = p1.z;
  int st = p1.w;
  if (blk * TJ_ROWS >= nodes * a.G) return;
  const bool live = m < nodes * a.G;
  // the rows' unit (one for all of them: blocks do not cross units), and the
  // CTAs that hold its first and last tile
  const long long u0 = before + (long long)(blk * TJ_ROWS / a.rows * a.nkv + kvh) * padded, u1 = u0 + tiles;
  const int b0 = st == 0 ? (int)div_ll(u0, share) : 0, b1 = st == 0 ? (int)div_ll(u1 - 1, share) : 0;
  if (a.part_err != nullptr && st == 0) {  // CTAs that gave up on a wait
    bool gave_up = false;
    for (int b = b0 + (int)threadIdx.x; b <= b1; b += TJ_THREADS) gave_up |= __ldcg(a.part_err + b) != 0u;
    if (__syncthreads_or(gave_up)) {
      st |= SPEC_ST_TIMEOUT;
      if (threadIdx.x == 0) atomicOr(a.status + s, SPEC_ST_TIMEOUT);
    }
  }
  if (st == 0 && b0 == b1) return;  // whole: written by its CTA
  for (int d0 = 8 * (SPLIT ? slice : slice * TJ_WARPS + warp); d0 < HD; d0 += 8 * (SPLIT ? slices : slices * TJ_WARPS)) {
    uint4* dst = reinterpret_cast<uint4*>(
        a.out + (((int64_t)s * a.nt + node) * a.nq + kvh * a.G + (m - node * a.G)) * HD + d0);
    if (st != 0) {
      if (live) *dst = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
      continue;
    }
    const float4* po = reinterpret_cast<const float4*>(a.part_o) + (size_t)(d0 / 4) * a.rows + r;
    const size_t piece = (size_t)a.rows * (HD / 4);
    constexpr int U = 8;
    const int per = SPLIT ? (b1 - b0 + TJ_WARPS) / TJ_WARPS : b1 + 1 - b0;  // pieces of a warp
    const int w0 = SPLIT ? b0 + warp * per : b0, w1 = min(b1 + 1, w0 + per);
    float mx = -INFINITY, l = 0.0f, o[8] = {};
    for (int bb = w0; bb < w1; bb += U) {
      float2 ml[U];
      float4 v[U][2];
#pragma unroll
      for (int j = 0; j < U; j++) {
        ml[j] = make_float2(-INFINITY, 0.0f);
        v[j][0] = v[j][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (bb + j < w1 && live) {
          // piece of CTA b: its first, unless it began in front of the unit
          const size_t slot = (size_t)(bb + j) * 2 + (share * (bb + j) < u0 ? 1 : 0);
          ml[j] = __ldcg(a.part_ml + slot * a.rows + r);
          v[j][0] = __ldcg(po + slot * piece);
          v[j][1] = __ldcg(po + slot * piece + a.rows);
        }
      }
      float m2 = mx;
#pragma unroll
      for (int j = 0; j < U; j++) m2 = fmaxf(m2, ml[j].x);
      const float ref = m2 == -INFINITY ? 0.0f : m2, alpha = exp2_fast(mx - ref);
      mx = m2;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < 8; d++) o[d] *= alpha;
#pragma unroll
      for (int j = 0; j < U; j++) {
        const float w = exp2_fast(ml[j].x - ref);
        l = fmaf(ml[j].y, w, l);
        o[0] = fmaf(v[j][0].x, w, o[0]);
        o[1] = fmaf(v[j][0].y, w, o[1]);
        o[2] = fmaf(v[j][0].z, w, o[2]);
        o[3] = fmaf(v[j][0].w, w, o[3]);
        o[4] = fmaf(v[j][1].x, w, o[4]);
        o[5] = fmaf(v[j][1].y, w, o[5]);
        o[6] = fmaf(v[j][1].z, w, o[6]);
        o[7] = fmaf(v[j][1].w, w, o[7]);
      }
    }
    if (SPLIT) {
#pragma unroll
      for (int d = 0; d < 8; d++) s_o[warp][d][lane] = o[d];
      s_ml[warp][lane] = make_float2(mx, l);
      __syncthreads();
      if (warp != 0) return;
#pragma unroll
      for (int w = 1; w < TJ_WARPS; w++) mx = fmaxf(mx, s_ml[w][lane].x);
      l = 0.0f;
#pragma unroll
      for (int d = 0; d < 8; d++) o[d] = 0.0f;
#pragma unroll
      for (int w = 0; w < TJ_WARPS; w++) {
        const float2 ml = s_ml[w][lane];
        const float f = exp2_fast(ml.x - mx);  // mx is finite: every row sees itself
        l = fmaf(ml.y, f, l);
#pragma unroll
        for (int d = 0; d < 8; d++) o[d] = fmaf(s_o[w][d][lane], f, o[d]);
      }
    }
    const float inv = 1.0f / l;
    if (live)
      *dst = make_uint4(pack_f16(o[0] * inv, o[1] * inv), pack_f16(o[2] * inv, o[3] * inv),
                        pack_f16(o[4] * inv, o[5] * inv), pack_f16(o[6] * inv, o[7] * inv));
  }
}

// Query rows of a unit.  Up to 32 rows run on the mma.sync kernel, more on
// the tcgen05 one with 64, 128 or 256 that share one read of the cache.
int rows_of(int M) {
  return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
}
bool on_tc(int rows) { return rows >= 64; }

template <int HD, int MT>
cudaError_t launch_shape(const TreeArgs& a, int n_cta, cudaStream_t st) {
  return launch_dependent(tree_attn_kernel<HD, MT>, n_cta + 1, TT_THREADS, Shape<HD, MT>::SMEM, st, a);
}

template <int HD>
cudaError_t launch_join(const TreeArgs& a, int n_cta, cudaStream_t st) {
  const int blocks = (a.nt * a.G + TJ_ROWS - 1) / TJ_ROWS;
  const long long units = (long long)a.n_seq * blocks * a.nkv;
  const bool split = units * 8 <= n_cta;
  // (a slice of 32 dimensions a CTA as long as those are resident at once, eight an SM)
  const int slices = split ? HD / 8 : units * (HD / 32) <= 8 * device_sms() ? HD / 32 : 1;
  return launch_dependent(split ? tree_join_kernel<HD, true> : tree_join_kernel<HD, false>, (size_t)(units * slices),
                          32 * join_warps(split), 0, st, a, blocks, slices);
}

template <int HD>
int launch_hd(const TreeArgs& a, int n_cta, cudaStream_t st) {
  cudaError_t e = on_tc(a.rows)  ? tree_tc_launch(a, HD, n_cta, st)
                  : a.rows == 16 ? launch_shape<HD, 1>(a, n_cta, st)
                                 : launch_shape<HD, 2>(a, n_cta, st);
  if (e == cudaSuccess) e = launch_join<HD>(a, n_cta, st);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("tree attention: ") + cudaGetErrorString(e));
  return SPEC_OK;
}

template <int HD, int MT>
void init_shape() {
  cudaFuncSetAttribute(tree_attn_kernel<HD, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)Shape<HD, MT>::SMEM);
}

// The CTAs with tiles: what is resident, but for the one that plans.
int tree_ctas(int hd, int rows) { return std::max(1, (on_tc(rows) ? 1 : resident(hd, rows)) * device_sms() - 1); }

// Budget of the calling thread's calls for the first wait of a CTA (tree_set_wait_budget).
thread_local int t_wait_tries = LIN_WAIT_TRIES;

}  // namespace

int tree_check(const spec_pages* kv, int n_seq, int nt, int n_q_heads) {
  int rc = check_pages(kv, true);
  if (rc != SPEC_OK) return rc;
  if (kv->head_dim != 64 && kv->head_dim != 128)
    return fail(SPEC_E_UNSUPPORTED, "tree attention supports head_dim 64 or 128");
  if (n_seq < 1 || nt < 1 || nt > SPEC_MAX_TREE)
    return fail(SPEC_E_SHAPE, "n_seq >= 1 and nt in [1, 64] required");
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads != 0)
    return fail(SPEC_E_SHAPE, "n_q_heads must be a positive multiple of n_kv_heads");
  if ((int64_t)kv->max_pages * kv->page_size > INT32_MAX - 2 * TT_KEYS)
    return fail(SPEC_E_SHAPE, "max_pages * page_size must stay below 2^31 - 128 positions");
  if (n_q_heads / kv->n_kv_heads > 4096)
    return fail(SPEC_E_SHAPE, "more than 4096 query heads a kv head");
  if ((double)n_seq * nt * n_q_heads * (kv->head_dim / 8) > INT32_MAX) return fail(SPEC_E_SHAPE, "n_seq * nt * n_q_heads too large");
  return SPEC_OK;
}

cudaError_t tree_join_launch(const TreeArgs& a, int hd, int n_cta, cudaStream_t st) {
  return hd == 128 ? launch_join<128>(a, n_cta, st) : launch_join<64>(a, n_cta, st);
}

void tree_set_wait_budget(int tries) { t_wait_tries = tries; }

void tree_init_attrs() {
  init_shape<64, 1>();
  init_shape<64, 2>();
  init_shape<128, 1>();
  init_shape<128, 2>();
  tree_tc_init_attrs();
}

int tree_workspace(const spec_pages* kv, int n_seq, int nt, int n_q_heads, size_t* bytes) {
  const int rc = tree_check(kv, n_seq, nt, n_q_heads);
  if (rc != SPEC_OK) return rc;
  const int rows = rows_of(nt * (n_q_heads / kv->n_kv_heads));
  *bytes = tree_scratch(kv->head_dim, rows, tree_ctas(kv->head_dim, rows), n_seq);
  return SPEC_OK;
}

size_t tree_scratch(int hd, int rows, int n_cta, int n_seq) {
  const size_t n = n_cta, r = rows;
  return n * 2 * r * (sizeof(float) * hd + sizeof(float2)) + (n * sizeof(uint32_t) + 15) / 16 * 16 +
         (size_t)n_seq * sizeof(TreePlan);
}

void tree_fill(TreeArgs& a, const spec_pages* kv, int layer, const spec_tree* t, const uint16_t* q, int64_t q_stride,
               const uint16_t* k_new, const uint16_t* v_new, int64_t kv_stride, uint16_t* out, void* workspace,
               int32_t* status, int rows, int tile_shift, int n_cta, bool bounded_waits) {
  a.k = reinterpret_cast<const __half*>(kv->k) + (int64_t)layer * kv->layer_stride;
  a.v = reinterpret_cast<const __half*>(kv->v) + (int64_t)layer * kv->layer_stride;
  a.table = kv->table;
  a.len = kv->len;
  a.n_slots = kv->n_slots;
  a.max_pages = kv->max_pages;
  a.n_pages = kv->n_pages;
  a.nkv = kv->n_kv_heads;
  a.page_size = kv->page_size;
  a.page_shift = -1;
  for (int b = 0; b < 31; b++)
    if (kv->page_size == 1 << b) a.page_shift = b;
  a.slots = t->slots;
  a.parents = t->parents;
  a.n_nodes = t->n_nodes;
  a.n_seq = t->n_seq;
  a.nt = t->nt;
  a.nq = t->n_q_heads;
  a.G = t->n_q_heads / kv->n_kv_heads;
  a.g_inv = (uint32_t)(((1ull << 32) + a.G - 1) / a.G);
  a.window = t->window;
  a.sinks = t->sinks;
  a.scale_log2 = (t->scale != 0.0f ? t->scale : 1.0f / sqrtf((float)kv->head_dim)) * 1.4426950408889634f;
  a.q = reinterpret_cast<const __half*>(q);
  a.q_stride = q_stride != 0 ? q_stride : (int64_t)a.nq * kv->head_dim;
  a.k_new = reinterpret_cast<const __half*>(k_new);
  a.v_new = reinterpret_cast<const __half*>(v_new);
  a.kv_stride = kv_stride != 0 ? kv_stride : (int64_t)a.nkv * kv->head_dim;
  a.out = reinterpret_cast<__half*>(out);
  a.status = status;
  a.rows = rows;
  a.tile_shift = tile_shift;
  a.part_o = reinterpret_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)n_cta * 2 * rows * kv->head_dim);
  uint32_t* err = reinterpret_cast<uint32_t*>(a.part_ml + (size_t)n_cta * 2 * rows);
  a.part_err = bounded_waits ? err : nullptr;
  a.wait_tries = t_wait_tries;
  a.plan = reinterpret_cast<TreePlan*>(err + ((size_t)n_cta + 3) / 4 * 4);
  a.k_qs = a.v_qs = nullptr;
  a.k_scales = a.v_scales = nullptr;
}

int launch_tree(const spec_pages* kv, int layer, const spec_tree* t, const uint16_t* q,
                int64_t q_stride, const uint16_t* k_new, const uint16_t* v_new, int64_t kv_stride,
                uint16_t* out, void* workspace, int32_t* status, cudaStream_t st) {
  TreeArgs a;
  const int rows = rows_of(t->nt * (t->n_q_heads / kv->n_kv_heads)), n_cta = tree_ctas(kv->head_dim, rows);
  tree_fill(a, kv, layer, t, q, q_stride, k_new, v_new, kv_stride, out, workspace, status, rows,
            on_tc(rows) ? TREE_TC_SHIFT : TT_SHIFT, n_cta, on_tc(rows));
  return kv->head_dim == 128 ? launch_hd<128>(a, n_cta, st) : launch_hd<64>(a, n_cta, st);
}
