// tree_attn_tc.cu -- tree attention for many query rows a kv head, on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// With up to 64 nodes and a GQA group of 4 to 8, one (sequence, kv head) has
// 64 to 512 query rows: 2 x rows flops per byte of the cache, which
// mma.sync (about a quarter of tcgen05's rate) cannot keep up with the HBM.
// One CTA per SM holds 128 or 256 rows against tiles of 128 positions, in
// roles that only meet at mbarriers:
//   warps 8-11   gather the positions' rows through the page table, two
//                warps K's and two V's, into rings of two and three
//                128-position buffers (16-byte cp.async, written in the MMA's
//                128-byte-swizzled layout; K as a K-major operand, V as an
//                MN-major one, so that neither is transposed)
//   warps 12, 13 issue S_j = Q_j K^T and O_j += P_j V, one stream each
//   warps 0-3, 4-7  two streams j = 0, 1: a thread owns a row; it reads its
//                scores from tensor memory, keeps the running maximum and sum
//                in fp32 (log2 domain) and writes P back over the scores as a
//                pair of fp16 numbers, hi and lo, which the MMA takes as its A
//                operands one after the other
// The streams keep the tensor core busy while the other one is in its
// softmax: with 256 rows they are the two row halves of every tile, with up
// to 128 they take the even and the odd tiles of the same rows, each with its
// own (max, sum, O), joined at the end.  With up to 64 the rows stand in the
// Q tile twice, stream 0 has those of lanes 0-63 and stream 1 those of lanes
// 64-127, so that the four SM sub-partitions share the softmax evenly.
//
// O is only rescaled when a row's maximum has grown by more than 2^3 since
// the last time (the weights may exceed 1 until then), so the accumulator in
// tensor memory is hardly ever touched by the softmax.  2^12 is multiplied into
// weights and sum alike, which keeps them below 2^15 and, with it, inside
// fp16's range: of a weight w the pair holds all but 2^-20 w + 2^-36, so that
// keys far below a row's largest are there, too (of n keys 20 nats below it, a
// sum n e^-20 in front of the rounding of the output).  One fp16 number would
// leave out 2^-11 w, as much again as the rounding of the output.
//
// Measured: 2 x 16 nodes over 131071 positions (32 heads over 8 of 128, 1.07
// GB) 181 us, 5.9 TB/s, 87% of the copy bandwidth: the memory.  4 x 63 nodes
// over 8191 positions 57 us, of which about 8 are the start (cut, tensor
// memory, page lookups, first tiles), 8 the end and the joining kernel, and
// 2.4 a tile of 128 positions x 256 rows: a stream's own chain of S, softmax
// and P V (the products of both streams alone take 1.9).  12 x 16 nodes over
// 512 positions, five tiles a unit and a unit a CTA, 24.6 us: start and end.
// With weights of one fp16 number these were 181, 48 and 24.  Not kept: the high
// parts' product under the forming of the low ones (57 -> 56 us), rings of three
// K and two V buffers (57 -> 59; 4 x 63 nodes each).
#include <math.h>

#include "common.cuh"
#include "tc_ops.cuh"
#include "tree_attn.cuh"

namespace {

constexpr int TC_SHIFT = TREE_TC_SHIFT, TC_KEYS = 1 << TC_SHIFT;
constexpr int K_RING = 2, V_RING = 3, TC_RING = K_RING + V_RING;
constexpr int TC_THREADS = 512;
constexpr int PROD_WARP = 8, MMA_WARP = 12, ALLOC_WARP = 14;
constexpr int PROD_THREADS = 64;  // of K's loads, and of V's
// Registers a thread: the softmax keeps a row's 128 scores.  Both pairs of
// warpgroups together hold the 512 x 128 of the launch.
constexpr int REGS_SOFTMAX = 200, REGS_OTHER = 56;
constexpr float P_BIAS = 12.0f;  // log2 of the factor of weights and sum
constexpr float P_SLACK = 3.0f;  // growth of the maximum before O is rescaled
constexpr int P_LO = 64;         // columns from the weights' high parts to their low ones

template <int HD>
struct TcShape {
  static constexpr int TILE = TC_KEYS * HD * 2;  // bytes of a Q, K or V tile
  static constexpr int SUB = TC_KEYS * 128;      // bytes of its 64-dimension part
  static constexpr int RING_OFF = 2 * TILE;
  static constexpr int END = RING_OFF + TC_RING * TILE;
};

struct TcSmall {
  unsigned long long full[TC_RING], empty[TC_RING];
  unsigned long long q_full, drain[2];
  unsigned long long s_full[2], p_ready[2], o_done[2];
  unsigned long long bad[TC_RING][2];  // rows of a masked V tile with a non-finite chunk
  long long part[TC_THREADS / 32];
  Start at;
  uint32_t tmem;
  int abort;
  signed char depth[2][SPEC_MAX_TREE];
  float2 x_ml[2][128];
};
constexpr int SMALL_MAX = 3072;
static_assert(sizeof(TcSmall) <= SMALL_MAX, "behind the tiles");
template <int HD>
constexpr size_t tc_smem() {
  return (size_t)TcShape<HD>::END + SMALL_MAX;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float half_of(uint32_t v, int hi) {
  return __half2float(__ushort_as_half((unsigned short)(hi ? v >> 16 : v & 0xFFFFu)));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A 16-byte chunk of fp16 with an infinity or NaN in it.
__device__ __forceinline__ bool odd_chunk(const uint4& v) {
  auto odd = [](uint32_t x) { return (x & 0x7C00u) == 0x7C00u || (x & 0x7C000000u) == 0x7C000000u; };
  return odd(v.x) || odd(v.y) || odd(v.z) || odd(v.w);
}

// --- tensor memory -----------------------------------------------------------
#define TREE_REGS32(v)                                                                             \
  "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), \
      "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),    \
      "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),  \
      "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),  \
      "+r"(v[29]), "+r"(v[30]), "+r"(v[31])

// 32 columns of this thread's lane; the values are there after tm_wait_ld.
__device__ __forceinline__ void tm_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tm_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  asm volatile("" : TREE_REGS32(v));  // nothing that uses them moves up
}
__device__ __forceinline__ uint32_t tm_ld1(uint32_t taddr) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n tcgen05.wait::ld.sync.aligned;"
               : "=r"(v) : "r"(taddr) : "memory");
  return v;
}
__device__ __forceinline__ void tm_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// D += A B with A (fp16 pairs) in tensor memory.
__device__ __forceinline__ void tc_mma_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {  // the same lane each time
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0u;
}
// MN-major operand, 128-byte swizzle: 64 of the MN dimension are the 128
// contiguous bytes, 8 of the K dimension an atom of 1024 bytes (stride byte
// offset), `lead` bytes from one 64 of MN to the next (leading byte offset).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}

// --- two floats at a time ------------------------------------------------------
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// Bits [0, n) of 32.
__device__ __forceinline__ uint32_t low_bits(long long n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << (int)n) - 1u;
}

template <int HD, int ROWS>
__global__ void __launch_bounds__(TC_THREADS, 1) tree_attn_tc_kernel(const TreeArgs a) {
  using Sh = TcShape<HD>;
  constexpr bool TWO = ROWS == 256;
  constexpr int UNITS = HD / 8, CH = HD / 32;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sm0 = smem_u32(smem);
  TcSmall& sh = *reinterpret_cast<TcSmall*>(smem + Sh::END);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  grid_dep_begin();
  const int n_cta = gridDim.x - 1;
  if ((int)blockIdx.x == n_cta) {
    plan_sequences<TC_THREADS>(a, ROWS, TC_SHIFT, n_cta, sh.part, smem);
    return;
  }
  Start start;
  const long long my_tiles = find_range<TC_THREADS>(a, ROWS, TC_SHIFT, n_cta, sh.part, smem, &sh.at, start);
  if (my_tiles <= 0 || (sm0 & 1023u) != 0u) {  // no tiles (a base off the swizzle's atoms never happens)
    if (tid == 0) a.part_err[blockIdx.x] = my_tiles > 0;
    if (warp < 8) check_others<TC_THREADS>(a, ROWS, TC_SHIFT, n_cta, 8);
    return;
  }
  auto bar = [&](unsigned long long& b) { return smem_u32(&b); };
  if (tid == 0) {
    sh.at = start;
    for (int i = 0; i < TC_RING; i++) {
      mbar_init(bar(sh.full[i]), PROD_THREADS);
      mbar_init(bar(sh.empty[i]), TWO ? 2 : 1);  // the streams that read it
    }
    mbar_init(bar(sh.q_full), 256);
    for (int j = 0; j < 2; j++) {
      mbar_init(bar(sh.s_full[j]), 1);
      mbar_init(bar(sh.p_ready[j]), 128);
      mbar_init(bar(sh.o_done[j]), 1);
      mbar_init(bar(sh.drain[j]), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sh.abort = 0;
  }
  if (warp == ALLOC_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sh.tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;  // columns: S_0, S_1 (128 each; P_j over S_j), O_0, O_1
  volatile int* abort_flag = &sh.abort;
  // Every wait on another role is bounded; once one has given up the others
  // return at their first try.  The loads and the products then end there, the
  // softmax (whose warps meet at barriers of their own) runs to its end with
  // whatever is there.
  auto wait = [&](unsigned long long& b, uint32_t parity) {
    const bool ok = mbar_wait(smem_u32(&b), parity & 1u, LIN_WAIT_TRIES, abort_flag);
    if (!ok) *abort_flag = 1;
    return ok;
  };
  // Buffers and turns of K and V of the CTA's tile x.  Each has a ring of its
  // own: a barrier tells a phase from the next one only, and as the streams
  // run freely against each other, a loader may not leave out a phase of a
  // buffer.  V's are held longer than K's.
  struct Item {
    uint32_t slot, turn;
  };
  auto item_k = [](uint32_t x) { return Item{x % K_RING, x / K_RING}; };
  auto item_v = [](uint32_t x) { return Item{K_RING + x % V_RING, x / V_RING}; };

  // (out of shared memory: nothing is known about them, and kept in registers, here)
  int s = sh.at.s;
  long long off = sh.at.off;
  SeqInfo q = sh.at.q;
  uint32_t tile0 = 0, seg = 0;  // tiles and pieces before this one
  // what a piece is
  int t0 = 0, n = 0, kvh = 0, row0 = 0, M = 0;
  auto next_piece = [&](long long left) {
    while (off >= q.work()) {
      s++;
      off = 0;
      q = seq_info(a, s, ROWS, TC_SHIFT);
    }
    const int unit = (int)div_ll(off, q.tiles);
    t0 = (int)(off - (long long)unit * q.tiles);
    n = (int)min((long long)(q.tiles - t0), left);
    kvh = unit % a.nkv;
    row0 = unit / a.nkv * ROWS;
    M = q.m * a.G;
  };
  auto tile_base = [&](int t) { return (t < q.n_sink ? t : q.w_tile + t - q.n_sink) << TC_SHIFT; };
  auto tile_masked = [&](int t) {
    if (t == q.tiles - 1) return true;
    const int base = tile_base(t);
    return base + TC_KEYS > q.len ||
           (a.window > 0 && base + TC_KEYS > q.sinks && base < q.lo + SPEC_MAX_TREE);
  };

  if (warp >= PROD_WARP && warp < PROD_WARP + 4) {
    // ======================================================= the loads
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    const bool is_k = warp < PROD_WARP + 2;
    const int pw = warp & 1;                         // rows 64 pw .. 64 pw + 63 of a tile
    constexpr int RPP = 32 / UNITS, PASSES = 64 / RPP;  // rows a pass of the warp
    const int u = lane % UNITS, sub = lane / UNITS;
    // where this lane's chunk of row RPP p + sub goes: the swizzle repeats every 8 rows
    uint32_t dst8[8 / RPP];
#pragma unroll
    for (int p = 0; p < 8 / RPP; p++)
      dst8[p] = (uint32_t)((u >> 3) * Sh::SUB) + sw128_off(64 * pw + RPP * p + sub, u & 7);
    auto dst_off = [&](int p) { return dst8[p % (8 / RPP)] + (uint32_t)(p / (8 / RPP)) * 1024u; };
    const __half* pool = (is_k ? a.k : a.v) + u * 8;
    const __half* fresh = (is_k ? a.k_new : a.v_new) + u * 8;
    struct Rows {
      uint32_t at[2];  // cache rows of the tile's rows lane and lane + 32 of the warp's 64
    };
    auto lookup = [&](int t) {
      Rows x = {{~0u, ~0u}};
      if (t == q.tiles - 1) return x;
      const int base = tile_base(t) + 64 * pw + lane;
      const int32_t* row = a.table + (int64_t)q.slot * a.max_pages;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int pos = base + 32 * h;
        if (pos < q.len) {
          const int e = a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
          const int pg = row[e];
          if (pg >= 0 && pg < a.n_pages)
            x.at[h] = ((uint32_t)pg * a.nkv + kvh) * a.page_size + (uint32_t)(pos - e * a.page_size);
        }
      }
      return x;
    };
    bool go = true;
    for (long long left = my_tiles; left > 0 && go; left -= n, off += n, tile0 += n, seg++) {
      next_piece(left);
      // the rows of the next tile are looked up while this one waits for its buffer
      Rows next = lookup(t0);
      for (int i = 0; i < n; i++) {
        const int t = t0 + i;
        const Item item = is_k ? item_k(tile0 + i) : item_v(tile0 + i);
        const uint32_t slot = item.slot, buf = sm0 + Sh::RING_OFF + slot * Sh::TILE;
        const Rows x = next;
        if (i + 1 < n) next = lookup(t + 1);
        go = __all_sync(0xffffffffu, wait(sh.empty[slot], item.turn + 1));
        if (!go) break;
        if (t == q.tiles - 1) {
          const __half* src = fresh + (int64_t)s * a.nt * a.kv_stride + kvh * HD;
#pragma unroll 4
          for (int p = 0; p < PASSES; p++) {
            const int r = 64 * pw + RPP * p + sub;
            const bool ok = r < q.m;
            cp16(buf + dst_off(p), src + (ok ? r : 0) * a.kv_stride, ok);
          }
        } else {
#pragma unroll
          for (int p = 0; p < PASSES; p++) {
            const uint32_t at = __shfl_sync(0xffffffffu, x.at[p / (PASSES / 2)], (RPP * p + sub) & 31);
            const bool ok = at != ~0u;
            cp16(buf + dst_off(p), pool + (uint64_t)(ok ? at : 0u) * HD, ok);
          }
        }
        if (is_k || !tile_masked(t)) {
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(sh.full[slot])) : "memory");
          continue;
        }
        // a masked tile's V: chunks with infinities or NaN, which 0 * inf
        // would spread to rows that do not see them, are taken out here and
        // added by the rows that do
        asm volatile("cp.async.wait_all;" ::: "memory");
        unsigned long long bad = 0ull;
#pragma unroll 4
        for (int p = 0; p < PASSES; p++) {
          const uint32_t at = buf + dst_off(p);
          uint4 v;
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
          if (odd_chunk(v)) {
            bad |= 1ull << (RPP * p + sub);
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
        if (lane == 0) sh.bad[slot][pw] = bad;
        fence_proxy_async();
        mbar_arrive(bar(sh.full[slot]));
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= MMA_WARP) {
    // ======================================================= the products
    // One warp per stream, which runs as a whole and issues through one
    // elected lane: with warp-uniform control an MMA of 128 x 128 x 16 issues
    // in less than the 64 cycles that it takes, under a branch on the lane in
    // about 110.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    const int j = warp - MMA_WARP;
    if (j < 2) {
      // a negative scale: the scores' sign is turned by the MMA (negated A),
      // so that a row's maximum is the maximum of what is read
      const uint32_t id_s = idesc_f16(TC_KEYS) | (a.scale_log2 < 0.0f ? 1u << 13 : 0u);
      const uint32_t id_o = idesc_f16(HD) | (1u << 16);
      const uint64_t d_q = smem_desc_sw128(sm0 + (TWO ? j * Sh::TILE : 0));
      const uint64_t d_k = smem_desc_sw128(sm0 + Sh::RING_OFF), d_v = smem_desc_mn(sm0 + Sh::RING_OFF, Sh::SUB);
      const uint32_t tS = tmem + j * 128, tO = tmem + 256 + j * 128;
      uint32_t n_p = 0;  // the stream's tiles so far
      // Whether the products go on, by what this lane has waited for: once a
      // wait has given up nothing is issued any more, while the turns below are
      // still handed over.
      bool go = true;
      auto wait_item = [&](const Item& item) {
        go = wait(sh.full[item.slot], item.turn) && go;
        __syncwarp();
        fence_proxy_async();  // the copies, to the tensor core's proxy
      };
      auto scores = [&](const Item& item) {
        wait_item(item);
        const uint64_t dk = d_k + item.slot * (uint32_t)(Sh::TILE >> 4);
        if (elect_one() && go) {
#pragma unroll
          for (int kk = 0; kk < HD / 16; kk++) {
            const uint32_t o = ((kk >> 2) * Sh::SUB + (kk & 3) * 32) >> 4;
            tc_mma(tS, d_q + o, dk + o, id_s, kk > 0);
          }
          tc_commit(bar(sh.s_full[j]));
          tc_commit(bar(sh.empty[item.slot]));
        }
        __syncwarp();
      };
      // The streams take turns, each with its P V and its next S in one go: were
      // both streams' products mixed, both would wait for theirs, and then
      // both be in their softmax, with the tensor core idle.  These barriers
      // have no limit of their own, and need none: both warps go through the
      // same pieces and tiles whatever their bounded waits say, and meet
      // between two pieces, so that no barrier is arrived at twice.
      auto hand_over = [](int id) { asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory"); };
      auto take_over = [](int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); };
      constexpr int TURN_0_1 = 4, TURN_1_0 = 5, START_0_1 = 6, PIECE = 7;
      for (long long left = my_tiles; left > 0; left -= n, off += n, tile0 += n, seg++) {
        next_piece(left);
        const int step = TWO ? 1 : 2;
        int i = TWO ? 0 : j;
        if (seg > 0) take_over(PIECE);
        go = wait(sh.q_full, seg) && go;  // (without a tile, too: a phase each piece)
        __syncwarp();
        if (i >= n) continue;
        if (j == 1) take_over(START_0_1);
        scores(item_k(tile0 + i));
        if (j == 0 && (TWO || n > 1)) hand_over(START_0_1);
        for (; i < n; i += step) {
          const Item vi = item_v(tile0 + i);
          const uint64_t dv = d_v + vi.slot * (uint32_t)(Sh::TILE >> 4);
          wait_item(vi);
          go = wait(sh.p_ready[j], n_p++) && go;
          __syncwarp();
          tc_fence_after();
          if (j == 1 || i > 0) take_over(j == 1 ? TURN_0_1 : TURN_1_0);
          if (elect_one() && go) {
#pragma unroll 1  // (sixteen in a row take registers that this warp does not have)
            for (int lo = 0; lo <= P_LO; lo += P_LO)
#pragma unroll
              for (int kk = 0; kk < TC_KEYS / 16; kk++)
                tc_mma_ta(tO, tS + lo + 8 * kk, dv + ((kk * 2048) >> 4), id_o, 1u);
            tc_commit(bar(sh.empty[vi.slot]));
            if (i + step >= n) tc_commit(bar(sh.o_done[j]));  // the stream's last tile
          }
          __syncwarp();
          if (i + step < n) scores(item_k(tile0 + i + step));
          if (TWO ? j == 0 || i + 1 < n : i + 1 < n) hand_over(j == 0 ? TURN_0_1 : TURN_1_0);
        }
      }
      // the products that were issued have ended before this CTA's memory is
      // another's: with the full budget, whether a wait has given up or not
      if (elect_one()) tc_commit(bar(sh.drain[j]));
      __syncwarp();
      if (!mbar_wait(bar(sh.drain[j]), 0u, LIN_WAIT_TRIES)) *abort_flag = 1;
    }
    __syncwarp();
  } else {
    // ======================================================= the softmax
    check_others<TC_THREADS>(a, ROWS, TC_SHIFT, n_cta, 8);  // (here, as the first keys are on their way)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    const int j = warp >> 2, r = tid & 127;  // stream, lane of tensor memory
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + j * 128, tO = tmem + lanes + 256 + j * 128;
    const float scale = fabsf(a.scale_log2);
    uint32_t n_s = 0, n_o = 0;  // tiles and pieces of this stream so far
    for (long long left = my_tiles; left > 0; left -= n, off += n, tile0 += n, seg++) {
      next_piece(left);
      const int nj = TWO ? n : (n - j + 1) / 2;
      // this thread's row of the unit; its chunks of the q tile
      const int rr = ROWS == 64 ? r & 63 : ROWS == 128 ? r : 128 * j + r;
      const int m = row0 + rr;
      const bool in = m < M;
      const bool live = in && (ROWS != 64 || (r >> 6) == j);
      const int wr = 32 * (warp & 3);  // the warp's first lane
      const bool warp_live = ROWS == 64 ? (wr >> 6) == j && row0 + (wr & 63) < M
                                        : row0 + (TWO ? 128 * j : 0) + wr < M;
      const int node = in ? node_of(a, m) : 0, head = kvh * a.G + (in ? m - node * a.G : 0);
      {
        const __half* src = a.q + ((int64_t)s * a.nt + node) * a.q_stride + head * HD;
        constexpr int MINE = TWO ? UNITS : UNITS / 2;  // both groups share a tile of one stream's rows
        const int u0 = TWO ? 0 : j * MINE;
        const uint32_t qt = sm0 + (TWO ? j * Sh::TILE : 0);
#pragma unroll
        for (int x = 0; x < MINE; x++) {
          const int u = u0 + x;
          cp16(qt + (u >> 3) * Sh::SUB + sw128_off(r, u & 7), src + u * 8, in);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(sh.q_full)) : "memory");
      }
      if (nj > 0) {
        uint32_t z[32];
#pragma unroll
        for (int c = 0; c < 32; c++) z[c] = 0u;
#pragma unroll
        for (int c = 0; c < CH; c++) tm_st32(tO + 32 * c, z);
      }
      // the row's node's ancestors and position
      auto parent = [&](int i) {
        const int p = a.parents != nullptr ? a.parents[(int64_t)s * a.nt + i] : i - 1;
        return p < i ? p : -1;  // (a tree that is none is refused by the joining kernel)
      };
      unsigned long long anc = 1ull << node;
      int depth = 0;
      for (int p = parent(node); p >= 0; p = parent(p)) {
        anc |= 1ull << p;
        depth++;
      }
      const int pos = q.len + depth;
      if (a.window > 0) {  // of its ancestors, those within the window
        if (r < q.m) {
          int d = 0;
          for (int p = parent(r); p >= 0; p = parent(p)) d++;
          sh.depth[j][r] = (signed char)d;
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + j) : "memory");
        for (unsigned long long left = anc; left != 0ull; left &= left - 1ull) {
          const int i = __ffsll((long long)left) - 1, p = q.len + sh.depth[j][i];
          if (!(p < a.sinks || p > pos - a.window)) anc &= ~(1ull << i);
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + j) : "memory");
      }
      if (!live) anc = 0ull;
      __syncwarp();
      tm_wait_st();
      float mx = -INFINITY, sum = 0.0f;
      for (int c = 0; c < nj; c++) {
        const int i = TWO ? c : 2 * c + j, t = t0 + i;
        if (!mbar_wait(bar(sh.s_full[j]), n_s & 1u, n_s == 0 ? a.wait_tries : LIN_WAIT_TRIES, abort_flag)) *abort_flag = 1;
        n_s++;
        __syncwarp();
        tc_fence_after();
        if (warp_live) {
          const bool masked = tile_masked(t);
          uint32_t v[4][32];
#pragma unroll
          for (int b = 0; b < 4; b++) tm_ld32(tS + 32 * b, v[b]);
#pragma unroll
          for (int b = 0; b < 4; b++) tm_wait_ld(v[b]);
          if (masked) {
            const bool tree = t == q.tiles - 1;
            const int base = tree ? 0 : tile_base(t);
#pragma unroll
            for (int b = 0; b < 4; b++) {
              uint32_t ok;  // bits of the visible keys 32 b .. 32 b + 31
              if (tree) {
                ok = b == 0 ? (uint32_t)anc : b == 1 ? (uint32_t)(anc >> 32) : 0u;
              } else {
                const long long p0 = (long long)base + 32 * b;
                ok = low_bits(q.len - p0);
                if (a.window > 0)
                  ok &= low_bits(a.sinks - p0) | ~low_bits((long long)pos - a.window + 1 - p0);
              }
#pragma unroll
              for (int e = 0; e < 32; e++)
                if (!((ok >> e) & 1u)) v[b][e] = __float_as_uint(-INFINITY);
            }
          }
          // ---- the tile's maximum
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int b = 0; b < 4; b++)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              x[b] = fmaxf(x[b], fmaxf(__uint_as_float(v[b][e]), __uint_as_float(v[b][e + 1])));
          const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * scale;
          const bool grow = top > mx + P_SLACK || (mx == -INFINITY && top > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = grow ? exp2_fast(mx - top) : 1.0f;  // 0 at first
            if (grow) mx = top;
            sum *= alpha;
            if (c > 0) {
#pragma unroll 1
              for (int d = 0; d < CH; d++) {
                uint32_t o[32];
                tm_ld32(tO + 32 * d, o);
                tm_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tm_st32(tO + 32 * d, o);
              }
            }
          }
          // ---- the weights over the scores, as pairs of fp16: hi is the
          // ---- weight cut off behind its 11th bit, lo the rest
          const float shift = P_BIAS - (mx == -INFINITY ? 0.0f : mx);
          const float2 sc2 = make_float2(scale, scale), sh2 = make_float2(shift, shift);
          float2 l[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int b = 0; b < 4; b++) {
#pragma unroll
            for (int e0 = 0; e0 < 32; e0 += 16) {
              uint32_t hi[8], lo[8];
#pragma unroll
              for (int e = e0; e < e0 + 16; e += 2) {
                const float2 y = fma2(make_float2(__uint_as_float(v[b][e]), __uint_as_float(v[b][e + 1])), sc2, sh2);
                const float2 p = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                l[(e >> 1) & 1] = add2(l[(e >> 1) & 1], p);
                const float2 cut = make_float2(__uint_as_float(__float_as_uint(p.x) & P_CUT),
                                               __uint_as_float(__float_as_uint(p.y) & P_CUT));
                const float2 rest = fma2(cut, make_float2(-P_REST, -P_REST), p);
                hi[(e - e0) >> 1] = pack_f16(cut.x, cut.y);
                lo[(e - e0) >> 1] = pack_f16(rest.x, rest.y);
              }
              tm_st8(tS + 16 * b + (e0 >> 1), hi);
              tm_st8(tS + P_LO + 16 * b + (e0 >> 1), lo);
            }
          }
          l[0] = add2(l[0], l[1]);
          sum += l[0].x + l[0].y;
          tm_wait_st();
          if (masked) {
            const Item item = item_v(tile0 + i);
            const uint32_t slot = item.slot;
            wait(sh.full[slot], item.turn);
            __syncwarp();
            // (one lane's reading for the whole warp, and a row's place checked:
            // after a wait that has given up the marks may be another tile's)
            const unsigned long long bad[2] = {__shfl_sync(0xffffffffu, sh.bad[slot][0], 0),
                                               __shfl_sync(0xffffffffu, sh.bad[slot][1], 0)};
            if ((bad[0] | bad[1]) != 0ull) {
              const bool tree = t == q.tiles - 1;
#pragma unroll 1
              for (int b = 0; b < 2; b++)
#pragma unroll 1
                for (unsigned long long left = b == 0 ? bad[0] : bad[1]; left != 0ull; left &= left - 1ull) {
                  const int key = 64 * b + __ffsll((long long)left) - 1;
                  const float p = half_of(tm_ld1(tS + (key >> 1)), key & 1) + half_of(tm_ld1(tS + P_LO + (key >> 1)), key & 1);
                  const __half* src = a.v;
                  if (tree) {
                    if (key >= q.m) continue;
                    src = a.v_new + ((int64_t)s * a.nt + key) * a.kv_stride + kvh * HD;
                  } else {
                    const int at = tile_base(t) + key, e = at / a.page_size;
                    if (at >= q.len) continue;
                    const int pg = a.table[(int64_t)q.slot * a.max_pages + e];
                    if (pg < 0 || pg >= a.n_pages) continue;
                    src += (((int64_t)pg * a.nkv + kvh) * a.page_size + (at - e * a.page_size)) * HD;
                  }
#pragma unroll 1
                  for (int d = 0; d < CH; d++) {
                    uint32_t o[32];
                    tm_ld32(tO + 32 * d, o);
                    tm_wait_ld(o);
#pragma unroll
                    for (int y = 0; y < 4; y++) {
                      const uint4 vv = *reinterpret_cast<const uint4*>(src + 32 * d + 8 * y);
                      if (p > 0.0f && odd_chunk(vv)) {
                        const uint32_t ww[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                        for (int e = 0; e < 8; e++)
                          o[8 * y + e] = __float_as_uint(fmaf(p, half_of(ww[e >> 1], e & 1), __uint_as_float(o[8 * y + e])));
                      }
                    }
                    __syncwarp();
                    tm_st32(tO + 32 * d, o);
                    tm_wait_st();
                  }
                }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(bar(sh.p_ready[j]));
      }
      // ---- the end of the piece
      if (nj > 0) {
        wait(sh.o_done[j], n_o++);
        __syncwarp();
        tc_fence_after();
      }
      const bool whole = t0 == 0 && n == q.tiles;
      const size_t slot = (size_t)blockIdx.x * 2 + (seg > 0 ? 1 : 0);
      // this warp's part of the q tiles, free now, turns rows of lanes into
      // rows of memory: 32 rows x D dimensions of fp16, 16-byte chunks swizzled
      const uint32_t turn = sm0 + warp * 32 * HD * 2;
      auto put_whole = [&](auto&& chunk, int D, int dim0) {  // chunk(c): 8 dimensions of this lane's row
        const int cr = D / 8, sw = cr >= 8 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
        for (int c = 0; c < cr; c++) {
          const uint4 y = chunk(c);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(turn + lane * D * 2 + ((c ^ sw) << 4)),
                       "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
        }
        __syncwarp();
        const int row_e = live ? node * a.nq + head : -1;  // this lane's row of the sequence's output
#pragma unroll
        for (int p = 0; p < cr; p++) {
          const int row = p * (32 / cr) + lane / cr, c = lane % cr;
          const int e = __shfl_sync(0xffffffffu, row_e, row), sw2 = cr >= 8 ? row & 7 : (row >> 1) & 3;
          uint4 y;
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                       : "r"(turn + row * D * 2 + ((c ^ sw2) << 4)));
          if (e >= 0)
            *reinterpret_cast<uint4*>(a.out + ((int64_t)s * a.nt * a.nq + e) * HD + dim0 + 8 * c) = y;
        }
      };
      auto put_piece = [&](int d, const uint32_t (&o)[32]) {  // dimensions 32 d .. 32 d + 31
        if (!live) return;
        uint4* po = reinterpret_cast<uint4*>(a.part_o) + (slot * (HD / 4) + 8 * d) * ROWS + rr;
#pragma unroll
        for (int x = 0; x < 8; x++)
          po[x * ROWS] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
      };
      auto chunk_of = [](const uint32_t (&o)[32], int c, float inv) {
        auto f = [&](int e) { return __uint_as_float(o[8 * (c & 3) + e]) * inv; };
        return make_uint4(pack_f16(f(0), f(1)), pack_f16(f(2), f(3)), pack_f16(f(4), f(5)), pack_f16(f(6), f(7)));
      };
      if (TWO || n == 1) {  // the row's one stream
        if (warp_live && nj > 0) {
          const float inv = 1.0f / sum;
          uint32_t o[CH][32];
#pragma unroll
          for (int d = 0; d < CH; d++) tm_ld32(tO + 32 * d, o[d]);
#pragma unroll
          for (int d = 0; d < CH; d++) tm_wait_ld(o[d]);
          if (whole) {
            put_whole([&](int c) { return chunk_of(o[c >> 2], c, inv); }, HD, 0);
          } else {
#pragma unroll
            for (int d = 0; d < CH; d++) put_piece(d, o[d]);
            if (live) a.part_ml[slot * ROWS + rr] = make_float2(mx, sum);
          }
        }
        // before the next q tile: its loaders have read what they turned
        if (TWO)
          asm volatile("bar.sync %0, 128;" ::"r"(1 + j) : "memory");
        else
          asm volatile("bar.sync 3, 256;" ::: "memory");
      } else {
        // the streams exchange halves: stream j finishes dimensions
        // [j HD / 2, (j + 1) HD / 2) of every row and hands the others over
        // through the q tiles: x[dimension][row].  The other stream may be a
        // tile behind, with an S to come
        asm volatile("bar.sync 3, 256;" ::: "memory");
        float* x_out = reinterpret_cast<float*>(smem + j * Sh::TILE);
        const float* x_in = reinterpret_cast<const float*>(smem + (1 - j) * Sh::TILE);
        constexpr int XR = ROWS == 64 ? 64 : 128;
        uint4 y[CH * 2];
        if (warp_live) {
          sh.x_ml[j][rr] = make_float2(mx, sum);
#pragma unroll
          for (int d = 0; d < CH / 2; d++) {
            uint32_t o[32];
            tm_ld32(tO + 32 * ((1 - j) * (CH / 2) + d), o);
            tm_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 32; e++) x_out[(32 * d + e) * XR + rr] = __uint_as_float(o[e]);
          }
        }
        asm volatile("bar.sync 3, 256;" ::: "memory");
        if (warp_live) {
          const float2 other = sh.x_ml[1 - j][rr];
          const float m2 = fmaxf(mx, other.x), ref = m2 == -INFINITY ? 0.0f : m2;
          const float w_own = exp2_fast(mx - ref), w_other = exp2_fast(other.x - ref);
          sum = sum * w_own + other.y * w_other;
          const float inv = 1.0f / sum;
          if (live && !whole && j == 0) a.part_ml[slot * ROWS + rr] = make_float2(m2, sum);
#pragma unroll
          for (int d = 0; d < CH / 2; d++) {
            uint32_t o[32];
            tm_ld32(tO + 32 * (j * (CH / 2) + d), o);
            tm_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 32; e++)
              o[e] = __float_as_uint(fmaf(x_in[(32 * d + e) * XR + rr], w_other, __uint_as_float(o[e]) * w_own));
            if (!whole) {
              put_piece(j * (CH / 2) + d, o);
            } else {
#pragma unroll
              for (int c = 0; c < 4; c++) y[4 * d + c] = chunk_of(o, c, inv);
            }
          }
        }
        asm volatile("bar.sync 3, 256;" ::: "memory");  // both halves have been read
        if (whole) {
          if (warp_live) put_whole([&](int c) { return y[c]; }, HD / 2, j * (HD / 2));
          asm volatile("bar.sync 3, 256;" ::: "memory");  // before the next q tile
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == ALLOC_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  if (tid == 0) a.part_err[blockIdx.x] = sh.abort != 0 ? 1u : 0u;
}

template <int HD, int ROWS>
cudaError_t launch(const TreeArgs& a, int n_cta, cudaStream_t st) {
  return launch_dependent(tree_attn_tc_kernel<HD, ROWS>, n_cta + 1, TC_THREADS, tc_smem<HD>(), st, a);
}

template <int HD>
cudaError_t launch_rows(const TreeArgs& a, int n_cta, cudaStream_t st) {
  return a.rows == 64    ? launch<HD, 64>(a, n_cta, st)
         : a.rows == 128 ? launch<HD, 128>(a, n_cta, st)
                         : launch<HD, 256>(a, n_cta, st);
}

template <int HD, int ROWS>
void init() {
  cudaFuncSetAttribute(tree_attn_tc_kernel<HD, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)tc_smem<HD>());
}

}  // namespace

cudaError_t tree_tc_launch(const TreeArgs& a, int hd, int n_cta, cudaStream_t st) {
  return hd == 128 ? launch_rows<128>(a, n_cta, st) : launch_rows<64>(a, n_cta, st);
}

void tree_tc_init_attrs() {
  init<64, 64>();
  init<64, 128>();
  init<64, 256>();
  init<128, 64>();
  init<128, 128>();
  init<128, 256>();
}
