// block_attn.cu -- attention over selected blocks of a cache, in fp16 or in 4
// bits (spec_block_attn, spec_block_attn_q4).
//
// Every (node, kv head) has a list of its own, so a unit is one node's group of
// query heads: 4 to 16 rows, the N of key_warp.cuh's products.  A cluster of CTAs
// has a unit; the keys of its list, 16 (codes: 32) a step, are dealt to the
// cluster's warps, each with a ring of its own and no barrier on the way, and the
// node's path of new rows, at most 64 keys, to the last of them.  The warps'
// results are joined in the CTA, the CTAs' through distributed shared memory: no
// workspace, no second launch.  All rows of a unit see the same keys, so that
// nothing is masked but the end of the last block.
//
// Measured (32 heads over 8 of 128): one node over 64 blocks of 64 in fp16 (17 MB) 8.9 us:
// launch, list, page, four steps a warp, of which two are on their way at a time, the cluster's
// join; 8 x 1 such nodes (134 MB) 26 us, 12 x 8 nodes over 64 blocks of 32 (807 MB named, 593 read) 103: the DRAM 71%
// busy.  In 4 bits 8 x 1 node (38 MB) 16.6 us: two CTAs a unit, eight steps a warp, 12% of the
// SMs' warps; 12 x 8 nodes (226 MB named, 165 read) 53: the chain of q4_attn.cu, issue slots 54%
// used.
#include <climits>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "key_warp.cuh"

namespace {

struct BlockArgs {
  const uint8_t* k;  // the layer's rows of fp16, or codes
  const uint8_t* v;
  const __half* k_scales;
  const __half* v_scales;
  const int32_t* table;
  const int32_t* len;
  int n_slots, max_pages, n_pages, nkv, page_size, shift;  // shift: log2 of the block
  const int32_t* slots;
  const int32_t* parents;
  const int32_t* n_nodes;
  int n_seq, nt, nq, G, row_blocks, keep, ranks;
  int path_rows;  // rows of the region for the path
  float scale_log2;
  const int32_t* blocks;
  const __half* q;
  int64_t q_stride;
  const __half* k_new;
  const __half* v_new;
  int64_t kv_stride;
  __half* out;
  int32_t* status;
};

template <int HD, int NT, bool Q4>
struct BShape {
  static constexpr int ROWS = 8 * NT;
  // a step of fp16 rows is 8 KB, of codes 4.6
  static constexpr int WARPS = Q4 ? 8 : 4, THREADS = 32 * WARPS, STAGES = Q4 ? 2 : 3;
  static constexpr int KEYS = Q4 ? 32 : 16, KT = KEYS / 16;  // keys of a step
  static constexpr int ROW = Q4 ? HD / 2 : HD * 2;           // bytes
  static constexpr int SCALES = Q4 ? KEYS * (HD / 16) : 0;
  static constexpr int STAGE = 2 * (KEYS * ROW + SCALES);
  static constexpr int RING = STAGES * STAGE;  // of a warp
  using Join = JoinShape<HD, ROWS, WARPS>;
  static constexpr int PART_OFF = ((WARPS * RING > Join::EXCHANGE ? WARPS * RING : Join::EXCHANGE) + 127) / 128 * 128;
  static constexpr int Q_OFF = (PART_OFF + Join::PART + 127) / 128 * 128;
  static constexpr int SUM_OFF = Q_OFF + KeyWarp<HD, NT, Q4>::Q_BYTES;
  static constexpr int PATH_OFF = (SUM_OFF + (Q4 ? KeyWarp<HD, NT, Q4>::SUM_BYTES : 0) + 127) / 128 * 128;
  // behind it path_rows rows of k_new and of v_new, then the list (8 bytes a block)
  static size_t smem(int path_rows, int keep) { return PATH_OFF + (size_t)path_rows * HD * 4 + (size_t)keep * 8; }
};

template <int HD, int NT, bool Q4>
__global__ void __launch_bounds__((BShape<HD, NT, Q4>::THREADS)) block_attn_kernel(const BlockArgs a) {
  using Sh = BShape<HD, NT, Q4>;
  using KW = KeyWarp<HD, NT, Q4>;
  constexpr int ROWS = Sh::ROWS, STAGES = Sh::STAGES, KEYS = Sh::KEYS, KT = Sh::KT, UNITS = HD / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ signed char s_par[SPEC_MAX_TREE], s_path[SPEC_MAX_TREE];
  __shared__ int s_depth, s_used;
  grid_dep_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % a.ranks, unit = blockIdx.x / a.ranks;
  const int rb = unit % a.row_blocks, kvh = unit / a.row_blocks % a.nkv, row_id = unit / a.row_blocks;
  const int node = row_id / a.nkv % a.nt, s = row_id / a.nkv / a.nt;
  const int slot = a.slots[s], m = a.n_nodes != nullptr ? a.n_nodes[s] : a.nt;
  const int32_t* list = a.blocks + (int64_t)row_id * a.keep;
  if (m >= 0 && m <= a.nt && node >= m) return;  // (all of the cluster)
  int st = 0, len = 0;
  if (slot < 0 || slot >= a.n_slots) {
    st |= SPEC_ST_SLOT;
  } else {
    len = a.len[slot];
    if (len < 0 || len > a.max_pages * a.page_size) st |= SPEC_ST_PAGE;
  }
  if (m < 0 || m > a.nt) st |= SPEC_ST_TREE;
  const int h0 = kvh * a.G + rb * ROWS, rows = min(ROWS, a.G - rb * ROWS);  // query heads
  uint32_t sm0 = kw_smem(smem);
  uint2* entry = reinterpret_cast<uint2*>(smem + Sh::PATH_OFF + (size_t)a.path_rows * HD * 4);
  // ---- the list (first cache row of a block, its positions), the path
  int bits = 0;
  if (tid == 0) s_used = 0;
  if (st == 0) {
    if (tid < SPEC_MAX_TREE) {
      int p = -1;
      if (tid < m) {
        p = a.parents != nullptr ? a.parents[(int64_t)s * a.nt + tid] : tid - 1;
        if (p < -1 || p >= tid) bits |= SPEC_ST_TREE;
      }
      s_par[tid] = (signed char)((bits & SPEC_ST_TREE) != 0 ? -1 : p);
    }
    __syncthreads();
    int used = 0;
    for (int e = tid; e < a.keep; e += Sh::THREADS) {
      const int b = list[e];
      uint2 x = make_uint2(0u, 0u);
      if (b < -1 || (b >= 0 && ((int64_t)b << a.shift) >= len)) {
        bits |= SPEC_ST_BLOCK;
      } else if (b >= 0) {
        const int pos = b << a.shift, pe = pos / a.page_size, pg = a.table[(int64_t)slot * a.max_pages + pe];
        if (pg < 0 || pg >= a.n_pages) {
          bits |= SPEC_ST_PAGE;
        } else {
          x.x = ((uint32_t)pg * a.nkv + kvh) * a.page_size + (uint32_t)(pos - pe * a.page_size);
          x.y = min(1 << a.shift, len - pos);
          used = e + 1;
        }
      }
      entry[e] = x;
    }
    if (used > 0) atomicMax(&s_used, used);
    if (tid == 0) {
      int n = 0;
      for (int p = node; p >= 0; p = s_par[p]) s_path[n++] = (signed char)p;
      s_depth = n;
    }
    if (__syncthreads_or(bits))
      for (int b = 1; b <= SPEC_ST_BLOCK; b <<= 1)
        if (__syncthreads_or(bits & b)) st |= b;
  }
  if (rank == 0 && rb == 0 && tid == 0) a.status[row_id] = st;
  if (st != 0) {
    if (rank == 0)
      for (int e = tid; e < rows * UNITS; e += Sh::THREADS)
        *reinterpret_cast<uint4*>(a.out + (((int64_t)s * a.nt + node) * a.nq + h0 + e / UNITS) * HD + e % UNITS * 8) =
            make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
    return;
  }
  const int n_path = s_depth;
  const int steps = (int)((((int64_t)s_used << a.shift) + KEYS - 1) / KEYS);
  const int warps = a.ranks * Sh::WARPS, gw = rank * Sh::WARPS + warp;
  const int path_steps = (n_path + 15) / 16, my_path = warps - 1 - gw;  // this warp's sixteen of the path, and those behind
  const uint32_t ring = sm0 + warp * Sh::RING, qs = sm0 + Sh::Q_OFF, sums = sm0 + Sh::SUM_OFF;
  const uint32_t kn0 = sm0 + Sh::PATH_OFF, vn0 = kn0 + a.path_rows * HD * 2;

  // the cache row of key i of step u, ~0: none
  auto lookup = [&](int u) {
    uint32_t x = ~0u;
    const int64_t key = (int64_t)u * KEYS + (lane & (KEYS - 1));
    const int e = (int)(key >> a.shift), at = (int)key & ((1 << a.shift) - 1);
    if (u < steps && e < s_used) {
      const uint2 b = entry[e];
      if (at < (int)b.y) x = b.x + at;
    }
    return x;
  };
  auto load_step = [&](int stage, uint32_t at) {
    const uint32_t to = ring + stage * Sh::STAGE;
    if constexpr (Q4) {
      load_codes<HD>(to, at, a.shift >= 5, a.k, a.v, a.k_scales, a.v_scales);
    } else {
      constexpr int CH = Sh::ROW / 16, PER = 32 / CH;
      const int c = lane % CH;
#pragma unroll
      for (int i = 0; i < KEYS / PER; i++) {
        const int r = i * PER + lane / CH;
        const uint32_t x = __shfl_sync(0xffffffffu, at, r);
        const bool ok = x != ~0u;
        const uint64_t from = (uint64_t)(ok ? x : 0u) * Sh::ROW + c * 16;
        kw_copy<16>(to + f16_off<HD>(r, c), a.k + from, ok);
        kw_copy<16>(to + KEYS * Sh::ROW + f16_off<HD>(r, c), a.v + from, ok);
      }
    }
  };
  // the path's rows first: they are few, and their step comes last
  for (int p = my_path; p < path_steps && my_path < Sh::WARPS; p += warps) {
    const int64_t from = (int64_t)s * a.nt * a.kv_stride + kvh * HD;
    for (int e = lane; e < 16 * UNITS; e += 32) {
      const int i = 16 * p + e / UNITS, u = e % UNITS;
      const bool ok = i < n_path;
      const int64_t at = from + (ok ? s_path[i] : 0) * a.kv_stride + u * 8;
      kw_copy<16>(kn0 + f16_off<HD>(i, u), a.k_new + at, ok);
      kw_copy<16>(vn0 + f16_off<HD>(i, u), a.v_new + at, ok);
    }
  }
  uint32_t now[STAGES];
#pragma unroll
  for (int i = 0; i < STAGES - 1; i++) {
    now[i] = lookup(gw + i * warps);
    if (gw + i * warps < steps) load_step(i, now[i]);
    asm volatile("cp.async.commit_group;");
  }
  KW::put_queries(qs, sums, tid, Sh::THREADS, a.scale_log2 < 0.0f, [&](int r) -> const __half* {
    return r < rows ? a.q + ((int64_t)s * a.nt + node) * a.q_stride + (h0 + r) * HD : nullptr;
  });
  __syncthreads();
  KW kw;
  kw.begin();
  const int gk = kw.g;
  const float scale = fabsf(a.scale_log2);
  int stage = 0;
  for (int u = gw; u < steps; u += warps) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncwarp();
    const int ahead = u + (STAGES - 1) * warps, next = stage == 0 ? STAGES - 1 : stage - 1;
    now[STAGES - 1] = lookup(ahead);
    if (ahead < steps) load_step(next, now[STAGES - 1]);
    asm volatile("cp.async.commit_group;");
    const uint32_t ks = ring + stage * Sh::STAGE, vs = ks + KEYS * Sh::ROW, kss = vs + KEYS * Sh::ROW,
                   vss = kss + Sh::SCALES;
    float x[KT][NT][4];
    if constexpr (Q4)
      kw.template scores_q4<KT>(ks, kss, qs, sums, x);
    else
      kw.scores_f16(ks, qs, x[0]);
    const uint32_t there = __ballot_sync(0xffffffffu, now[0] != ~0u);
    if (there != 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < 2 * KT; i++)
        if (!(there >> (8 * i + gk) & 1))
#pragma unroll
          for (int n = 0; n < NT; n++) x[i >> 1][n][2 * (i & 1)] = x[i >> 1][n][2 * (i & 1) + 1] = -INFINITY;
    }
    kw.template weights<KT>(Q4 ? scale * KW::CODE_UNIT : scale, x);
#pragma unroll
    for (int i = 0; i < KT; i++) {
      if constexpr (Q4)
        kw.values_q4(vs + 16 * i * Sh::ROW, vss + 16 * i * (HD / 16), x[i]);
      else
        kw.values_f16(vs, x[i]);
    }
#pragma unroll
    for (int i = 0; i < STAGES - 1; i++) now[i] = now[i + 1];
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  for (int p = my_path; p < path_steps && my_path < Sh::WARPS; p += warps) {
    float x[1][NT][4];
    kw.scores_f16(kn0 + f16_off<HD>(16 * p, 0), qs, x[0]);
#pragma unroll
    for (int i = 0; i < 2; i++)
      if (16 * p + 8 * i + gk >= n_path)
#pragma unroll
        for (int n = 0; n < NT; n++) x[0][n][2 * i] = x[0][n][2 * i + 1] = -INFINITY;
    kw.template weights<1>(scale, x);
    kw.values_f16(vn0 + f16_off<HD>(16 * p, 0), x[0]);
  }
  __syncthreads();  // the rings have been read
  __half* out = a.out + (((int64_t)s * a.nt + node) * a.nq + h0) * HD;
  join_unit<Sh::WARPS>(kw, smem, Sh::PART_OFF, rank, a.ranks, rows,
            [&](int r, int u, const float (&acc)[8], float l) { put_row(out + r * HD + u * 8, acc, l); });
}

constexpr size_t SM_SMEM = 228 * 1024;     // of an SM
constexpr size_t FIXED_SMEM = 1024 + 256;  // of a CTA beside what its launch asks for: the system's, the static arrays
// CTAs of a unit, as long as every warp has two steps of the list: of fp16 as many as are
// resident, two an SM, up to 16 (one node over 64 blocks of 64: 8.9 us, with up to eight
// 9.9); of codes, with twice the warps, one an SM, up to eight (8 sequences of one node
// over 64 blocks of 64: 17.3 us, with half the warps 20.8), and of fp16 with the longest
// lists, too, where the shared memory holds one: sixteen SMs may be more than a GPC has.
template <int HD, int NT, bool Q4>
int launch_block(BlockArgs& a, double units, int block, cudaStream_t st) {
  using Sh = BShape<HD, NT, Q4>;
  const size_t smem = Sh::smem(a.path_rows, a.keep);
  const int64_t steps = ((int64_t)a.keep * block + Sh::KEYS - 1) / Sh::KEYS;
  const int fit = !Q4 && 2 * (smem + FIXED_SMEM) <= SM_SMEM ? 2 : 1;
  a.ranks = 1;
  while (a.ranks < 8 * fit && units * a.ranks * 2 <= fit * device_sms() && steps >= (int64_t)2 * Sh::WARPS * a.ranks * 2)
    a.ranks *= 2;
  if (units * a.ranks > INT32_MAX) return fail(SPEC_E_SHAPE, "n_seq * nt * n_q_heads too large");
  const cudaError_t e = launch_clusters(block_attn_kernel<HD, NT, Q4>, a, (size_t)units * a.ranks, Sh::THREADS, a.ranks,
                                        smem, st);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("block attention: ") + cudaGetErrorString(e));
  return SPEC_OK;
}
template <int HD, bool Q4>
int launch_block_rows(BlockArgs& a, double units, int NT, int block, cudaStream_t st) {
  return NT == 1 ? launch_block<HD, 1, Q4>(a, units, block, st) : launch_block<HD, 2, Q4>(a, units, block, st);
}

template <int HD, int NT, bool Q4>
void init_block() {
  cudaFuncSetAttribute(block_attn_kernel<HD, NT, Q4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)BShape<HD, NT, Q4>::smem(SPEC_MAX_TREE, SPEC_MAX_KEEP));
  cudaFuncSetAttribute(block_attn_kernel<HD, NT, Q4>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

}  // namespace

void block_attn_init_attrs() {
  init_block<64, 1, false>();
  init_block<64, 2, false>();
  init_block<128, 1, false>();
  init_block<128, 2, false>();
  init_block<64, 1, true>();
  init_block<64, 2, true>();
  init_block<128, 1, true>();
  init_block<128, 2, true>();
}

int launch_block_attn(const spec_pages* book, const BlockPlanes& planes, const spec_tree* t, int block, int n_keep,
                      const int32_t* blocks, const uint16_t* q, int64_t q_stride, const uint16_t* k_new,
                      const uint16_t* v_new, int64_t kv_stride, uint16_t* out, int32_t* status, cudaStream_t st) {
  BlockArgs a;
  const int hd = book->head_dim;
  const bool q4 = planes.k_scales != nullptr;
  a.k = planes.k;
  a.v = planes.v;
  a.k_scales = reinterpret_cast<const __half*>(planes.k_scales);
  a.v_scales = reinterpret_cast<const __half*>(planes.v_scales);
  a.table = book->table;
  a.len = book->len;
  a.n_slots = book->n_slots;
  a.max_pages = book->max_pages;
  a.n_pages = book->n_pages;
  a.nkv = book->n_kv_heads;
  a.page_size = book->page_size;
  a.shift = block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
  a.slots = t->slots;
  a.parents = t->parents;
  a.n_nodes = t->n_nodes;
  a.n_seq = t->n_seq;
  a.nt = t->nt;
  a.nq = t->n_q_heads;
  a.G = t->n_q_heads / book->n_kv_heads;
  const int NT = a.G <= 8 ? 1 : 2;
  a.row_blocks = (a.G + 8 * NT - 1) / (8 * NT);
  a.keep = n_keep;
  a.path_rows = (t->nt + 15) / 16 * 16;
  a.scale_log2 = (t->scale != 0.0f ? t->scale : 1.0f / sqrtf((float)hd)) * 1.4426950408889634f;
  a.blocks = blocks;
  a.q = reinterpret_cast<const __half*>(q);
  a.q_stride = q_stride != 0 ? q_stride : (int64_t)a.nq * hd;
  a.k_new = reinterpret_cast<const __half*>(k_new);
  a.v_new = reinterpret_cast<const __half*>(v_new);
  a.kv_stride = kv_stride != 0 ? kv_stride : (int64_t)a.nkv * hd;
  a.out = reinterpret_cast<__half*>(out);
  a.status = status;
  const double units = (double)t->n_seq * t->nt * a.nkv * a.row_blocks;
  return hd == 128 ? (q4 ? launch_block_rows<128, true>(a, units, NT, block, st)
                          : launch_block_rows<128, false>(a, units, NT, block, st))
                   : (q4 ? launch_block_rows<64, true>(a, units, NT, block, st)
                         : launch_block_rows<64, false>(a, units, NT, block, st));
}
