// tree_attn_tc.cu -- tree attention for many query rows a kv head, on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// With up to 64 nodes and a GQA group of 4 to 8, one (sequence, kv head) has
// 64 to 512 query rows: 2 x rows flops per byte of the cache, which
// mma.sync (about a quarter of tcgen05's rate) cannot keep up with the HBM.
// One CTA per SM holds 128 or 256 rows against tiles of 128 positions, in
// roles that only meet at mbarriers:
//   warps 8, 9   gather the positions' K and V rows through the page table
//                into a ring of five 128-position buffers (16-byte cp.async,
//                written in the MMA's 128-byte-swizzled layout; K as a
//                K-major operand, V as an MN-major one, so that neither is
//                transposed)
//   warp 10      one thread issues S_j = Q_j K^T and O_j += P_j V
//   warps 0-3, 4-7  two streams j = 0, 1: a thread owns a row; it reads its
//                scores from tensor memory, keeps the running maximum and sum
//                in fp32 (log2 domain) and writes P back as fp16, over the
//                scores, where the MMA takes it as its A operand
// The streams keep the tensor core busy while the other one is in its
// softmax: with 256 rows they are the two row halves of every tile, with up
// to 128 they take the even and the odd tiles of the same rows, each with its
// own (max, sum, O), joined at the end.
//
// O is only rescaled when a row's maximum has grown by more than 2^8 since
// the last time (the weights may exceed 1 until then, by less than fp16's
// range), so the accumulator in tensor memory is hardly ever touched by the
// softmax.  The weights are rounded once, to fp16, which costs an output half
// an fp16 step of its average |v|: 2^-11 relative, as the rounding of the
// output itself; a second MMA with the rounding errors (as the kernel for few
// rows does, which waits for the cache anyway) would make the tensor core the
// bound.  2^6 is multiplied into weights and sum alike, so that those of 2^-20
// are still normal numbers.
#include <math.h>

#include "common.cuh"
#include "tc_ops.cuh"
#include "tree_attn.cuh"

namespace {

constexpr int TC_SHIFT = TREE_TC_SHIFT, TC_KEYS = 1 << TC_SHIFT;
constexpr int TC_RING = 5;
constexpr int TC_THREADS = 384;
constexpr int PROD_WARP = 8, MMA_WARP = 10, ALLOC_WARP = 11;
constexpr int PROD_THREADS = 64;
constexpr float P_BIAS = 6.0f;   // log2 of the factor of weights and sum
constexpr float P_SLACK = 8.0f;  // growth of the maximum before O is rescaled

template <int HD>
struct TcShape {
  static constexpr int TILE = TC_KEYS * HD * 2;  // bytes of a Q, K or V tile
  static constexpr int SUB = TC_KEYS * 128;      // bytes of its 64-dimension part
  static constexpr int RING_OFF = 2 * TILE;
  static constexpr int END = RING_OFF + TC_RING * TILE;
};

struct TcSmall {
  unsigned long long full[TC_RING], empty[TC_RING];
  unsigned long long q_full, q_empty, drain;
  unsigned long long s_full[2], p_ready[2], o_done[2];
  unsigned long long bad[TC_RING][2];  // rows of a masked V tile with a non-finite chunk
  long long part[TC_THREADS / 32];
  long long off;
  int seq;
  uint32_t tmem;
  int abort;
  signed char depth[2][SPEC_MAX_TREE];
  float2 x_ml[128];
};
constexpr int SMALL_MAX = 2048;
static_assert(sizeof(TcSmall) <= SMALL_MAX, "behind the tiles");
template <int HD>
constexpr size_t tc_smem() {  // the tiles start at a multiple of 1024 bytes
  return (size_t)TcShape<HD>::END + SMALL_MAX + 1024;
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
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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
// MN-major operand, 128-byte swizzle: 64 of the MN dimension are the 128
// contiguous bytes, 8 of the K dimension an atom of 1024 bytes (stride byte
// offset), `lead` bytes from one 64 of MN to the next (leading byte offset).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}

// Bits [0, n) of 32.
__device__ __forceinline__ uint32_t low_bits(long long n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << (int)n) - 1u;
}

template <int HD, bool TWO>
__global__ void __launch_bounds__(TC_THREADS, 1) tree_attn_tc_kernel(const TreeArgs a) {
  using Sh = TcShape<HD>;
  constexpr int ROWS = TWO ? 256 : 128, UNITS = HD / 8, CH = HD / 32;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw0 = smem_u32(smem_raw), sm0 = (raw0 + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (sm0 - raw0);
  TcSmall& sh = *reinterpret_cast<TcSmall*>(smem + Sh::END);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_launch();  // the joining kernel may get ready
  const Range range = find_range<TC_THREADS>(a, ROWS, TC_SHIFT, sh.part, &sh.seq, &sh.off);
  const long long w0 = range.w0, w1 = range.w1;
  if (w0 >= w1) {
    if (tid == 0) a.part_err[blockIdx.x] = 0u;
    return;
  }
  auto bar = [&](unsigned long long& b) { return smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < TC_RING; i++) {
      mbar_init(bar(sh.full[i]), PROD_THREADS);
      mbar_init(bar(sh.empty[i]), 1);
    }
    mbar_init(bar(sh.q_full), PROD_THREADS);
    mbar_init(bar(sh.q_empty), 256);
    mbar_init(bar(sh.drain), 1);
    for (int j = 0; j < 2; j++) {
      mbar_init(bar(sh.s_full[j]), 1);
      mbar_init(bar(sh.p_ready[j]), 128);
      mbar_init(bar(sh.o_done[j]), 1);
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
  // Every wait is bounded; once one has given up the others return at their
  // first try, and all roles run to their ends with whatever is there.
  auto wait = [&](unsigned long long& b, uint32_t parity) {
    if (!mbar_wait(smem_u32(&b), parity & 1u, LIN_WAIT_TRIES, abort_flag)) *abort_flag = 1;
  };
  // The ring's order: K runs LA tiles ahead of V.
  constexpr int LA = TWO ? 1 : 2;
  auto item_k = [](int i) { return TWO ? 2 * i : (i == 0 ? 0 : 2 * i - 1); };
  auto item_v = [](int i, int n) { return TWO ? 2 * i + 1 : min(2 * i + 2, 2 * n - 1); };

  int s = sh.seq;
  long long off = sh.off;
  SeqInfo q = seq_info(a, s, ROWS, TC_SHIFT);
  uint32_t item0 = 0, seg = 0;  // ring items and pieces before this one
  // what a piece is
  int t0 = 0, n = 0, kvh = 0, row0 = 0, M = 0;
  auto next_piece = [&](long long w) {
    while (off >= q.work()) {
      s++;
      off = 0;
      q = seq_info(a, s, ROWS, TC_SHIFT);
    }
    const int unit = (int)(off / q.tiles);
    t0 = (int)(off % q.tiles);
    n = (int)min((long long)(q.tiles - t0), w1 - w);
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

  if (warp >= PROD_WARP && warp < PROD_WARP + 2) {
    // ======================================================= the loads
    const int pw = warp - PROD_WARP;                 // rows 64 pw .. 64 pw + 63 of a tile
    constexpr int RPP = 32 / UNITS, PASSES = 64 / RPP;  // rows a pass of the warp
    const int u = lane % UNITS, sub = lane / UNITS;
    auto dst_off = [&](int r) { return (uint32_t)((u >> 3) * Sh::SUB) + sw128_off(r, u & 7); };
    for (long long w = w0; w < w1; w += n, off += n, item0 += 2 * n, seg++) {
      next_piece(w);
      auto load = [&](bool is_k, int i, uint32_t item) {
        const uint32_t slot = item % TC_RING, buf = sm0 + Sh::RING_OFF + slot * Sh::TILE;
        const int t = t0 + i;
        const bool tree = t == q.tiles - 1, scan = !is_k && tile_masked(t);
        // this lane looks up rows lane and lane + 32 of the warp's 64
        uint32_t idx[2] = {~0u, ~0u};
        if (!tree) {
          const int base = tile_base(t);
          const int32_t* row = a.table + (int64_t)q.slot * a.max_pages;
#pragma unroll
          for (int j = 0; j < 2; j++) {
            const int pos = base + 64 * pw + 32 * j + lane;
            if (pos < q.len) {
              const int e = a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
              const int pg = __ldg(row + e);
              if (pg >= 0 && pg < a.n_pages)
                idx[j] = (uint32_t)((pg * (int64_t)a.nkv + kvh) * a.page_size + (pos - e * a.page_size));
            }
          }
        }
        wait(sh.empty[slot], (item / TC_RING) + 1);
        const __half* src = is_k ? (tree ? a.k_new : a.k) : (tree ? a.v_new : a.v);
#pragma unroll 8
        for (int p = 0; p < PASSES; p++) {
          const int r = RPP * p + sub;
          bool ok;
          int64_t at;
          if (tree) {
            ok = 64 * pw + r < q.m;
            at = ((int64_t)s * a.nt + (ok ? 64 * pw + r : 0)) * a.kv_stride + kvh * HD;
          } else {
            const uint32_t x = __shfl_sync(0xffffffffu, p < PASSES / 2 ? idx[0] : idx[1], r & 31);
            ok = x != ~0u;
            at = ok ? (int64_t)x * HD : 0;
          }
          cp16(buf + dst_off(64 * pw + r), src + at + u * 8, ok);
        }
        if (!scan) {
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(sh.full[slot])) : "memory");
          return;
        }
        // a masked tile's V: chunks with infinities or NaN, which 0 * inf
        // would spread to rows that do not see them, are taken out here and
        // added by the rows that do
        asm volatile("cp.async.wait_all;" ::: "memory");
        unsigned long long bad = 0ull;
        for (int p = 0; p < PASSES; p++) {
          const uint32_t at = buf + dst_off(64 * pw + RPP * p + sub);
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
      };
      for (int i = 0; i < min(LA, n); i++) load(true, i, item0 + item_k(i));
      wait(sh.q_empty, seg + 1);
      for (int e = tid - PROD_WARP * 32; e < ROWS * UNITS; e += PROD_THREADS) {
        const int r = e / UNITS, uu = e % UNITS, m = row0 + r;
        const bool ok = m < M;
        const int node = ok ? m / a.G : 0, h = kvh * a.G + (ok ? m % a.G : 0);
        cp16(sm0 + (r >> 7) * Sh::TILE + (uu >> 3) * Sh::SUB + sw128_off(r & 127, uu & 7),
             a.q + ((int64_t)s * a.nt + node) * a.q_stride + h * HD + uu * 8, ok);
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(sh.q_full)) : "memory");
      for (int i = 0; i < n; i++) {
        load(false, i, item0 + item_v(i, n));
        if (i + LA < n) load(true, i + LA, item0 + item_k(i + LA));
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == MMA_WARP) {
    // ======================================================= the products
    if (lane == 0) {
      const uint32_t id_s = idesc_f16(TC_KEYS), id_o = idesc_f16(HD) | (1u << 16);
      uint32_t n_p[2] = {0, 0};  // tiles of each stream so far
      for (long long w = w0; w < w1; w += n, off += n, item0 += 2 * n, seg++) {
        next_piece(w);
        auto scores = [&](int j, uint32_t item) {
          const uint32_t kb = sm0 + Sh::RING_OFF + item % TC_RING * Sh::TILE, qb = sm0 + (TWO ? j * Sh::TILE : 0);
#pragma unroll
          for (int kk = 0; kk < HD / 16; kk++) {
            const uint32_t o = (kk >> 2) * Sh::SUB + (kk & 3) * 32;
            tc_mma(tmem + j * 128, smem_desc_sw128(qb + o), smem_desc_sw128(kb + o), id_s, kk > 0);
          }
          tc_commit(bar(sh.s_full[j]));
        };
        auto output = [&](int j, uint32_t item) {
          const uint32_t vb = sm0 + Sh::RING_OFF + item % TC_RING * Sh::TILE;
#pragma unroll
          for (int kk = 0; kk < TC_KEYS / 16; kk++)
            tc_mma_ta(tmem + 256 + j * 128, tmem + j * 128 + 8 * kk, smem_desc_mn(vb + kk * 2048, Sh::SUB),
                      id_o, 1u);
        };
        auto wait_item = [&](uint32_t item) {
          wait(sh.full[item % TC_RING], item / TC_RING);
          fence_proxy_async();  // the copies, to the tensor core's proxy
        };
        auto release = [&](uint32_t item) { tc_commit(bar(sh.empty[item % TC_RING])); };
        wait(sh.q_full, seg);
        fence_proxy_async();
        if (TWO) {
          const uint32_t k0 = item0 + item_k(0);
          wait_item(k0);
          scores(0, k0);
          scores(1, k0);
          release(k0);
        } else {
          for (int i = 0; i < min(2, n); i++) {
            const uint32_t ki = item0 + item_k(i);
            wait_item(ki);
            scores(i, ki);
            release(ki);
          }
        }
        for (int i = 0; i < n; i++) {
          const uint32_t vi = item0 + item_v(i, n), kn = item0 + item_k(i + LA);
          wait_item(vi);
          for (int j = TWO ? 0 : i & 1; j < (TWO ? 2 : (i & 1) + 1); j++) {
            wait(sh.p_ready[j], n_p[j]++);
            tc_fence_after();
            output(j, vi);
            if (i + LA >= n) tc_commit(bar(sh.o_done[j]));  // the stream's last tile
            if (!TWO || j == 1) release(vi);
            if (i + LA < n) {
              if (!TWO || j == 0) wait_item(kn);
              scores(j, kn);
              if (!TWO || j == 1) release(kn);
            }
          }
        }
      }
      tc_commit(bar(sh.drain));
      wait(sh.drain, 0);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ======================================================= the softmax
    const int j = warp >> 2, r = tid & 127;  // stream, row of its 128
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + j * 128, tO = tmem + lanes + 256 + j * 128;
    const bool neg = a.scale_log2 < 0.0f;
    uint32_t n_s = 0, n_o = 0;  // tiles and pieces of this stream so far
    for (long long w = w0; w < w1; w += n, off += n, item0 += 2 * n, seg++) {
      next_piece(w);
      const int nj = TWO ? n : (n - j + 1) / 2;
      const int m = row0 + (TWO ? 128 * j : 0) + r;
      const bool live = m < M;
      const bool warp_live = row0 + (TWO ? 128 * j : 0) + 32 * (warp & 3) < M;
      // this row's node, its ancestors, its position
      const int node = live ? m / a.G : 0;
      auto parent = [&](int i) {
        const int p = a.parents != nullptr ? __ldg(a.parents + (int64_t)s * a.nt + i) : i - 1;
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
      float mx = -INFINITY, sum = 0.0f;
      __syncwarp();
      if (nj > 0) {
        uint32_t z[32];
#pragma unroll
        for (int c = 0; c < 32; c++) z[c] = 0u;
#pragma unroll
        for (int c = 0; c < CH; c++) tm_st32(tO + 32 * c, z);
        tm_wait_st();
      }
      for (int c = 0; c < nj; c++) {
        const int i = TWO ? c : 2 * c + j, t = t0 + i;
        wait(sh.s_full[j], n_s++);
        __syncwarp();
        tc_fence_after();
        if (warp_live) {
          const bool tree = t == q.tiles - 1, masked = tile_masked(t);
          const int base = tree ? 0 : tile_base(t);
          // bits of the visible keys 32 b .. 32 b + 31
          auto seen = [&](int b) -> uint32_t {
            if (tree) return b == 0 ? (uint32_t)anc : b == 1 ? (uint32_t)(anc >> 32) : 0u;
            const long long p0 = (long long)base + 32 * b;
            uint32_t v = low_bits(q.len - p0);
            if (a.window > 0) v &= low_bits(a.sinks - p0) | ~low_bits((long long)pos - a.window + 1 - p0);
            return v;
          };
          uint32_t v[2][32];
          const float hidden = neg ? INFINITY : -INFINITY;  // before the scale
          // ---- the tile's maximum
          float best = hidden;
          tm_ld32(tS, v[0]);
#pragma unroll
          for (int b = 0; b < 4; b++) {
            tm_wait_ld(v[b & 1]);
            if (b < 3) tm_ld32(tS + 32 * (b + 1), v[(b + 1) & 1]);
            if (masked) {
              const uint32_t ok = seen(b);
#pragma unroll
              for (int e = 0; e < 32; e++)
                if (!((ok >> e) & 1u)) v[b & 1][e] = __float_as_uint(hidden);
            }
            float x[4] = {best, best, best, best};
            if (neg) {
#pragma unroll
              for (int e = 0; e < 32; e++) x[e & 3] = fminf(x[e & 3], __uint_as_float(v[b & 1][e]));
              best = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
            } else {
#pragma unroll
              for (int e = 0; e < 32; e++) x[e & 3] = fmaxf(x[e & 3], __uint_as_float(v[b & 1][e]));
              best = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            }
          }
          const float top = best * a.scale_log2;
          const bool grow = top > mx + P_SLACK || (mx == -INFINITY && top > -INFINITY);
          tm_ld32(tS, v[0]);
          if (__any_sync(0xffffffffu, grow)) {
            tm_wait_ld(v[0]);
            const float alpha = grow ? exp2_fast(mx - top) : 1.0f;  // 0 at first
            if (grow) mx = top;
            sum *= alpha;
            if (c > 0) {
#pragma unroll
              for (int d = 0; d < CH; d++) {
                tm_ld32(tO + 32 * d, v[1]);
                tm_wait_ld(v[1]);
#pragma unroll
                for (int e = 0; e < 32; e++) v[1][e] = __float_as_uint(__uint_as_float(v[1][e]) * alpha);
                tm_st32(tO + 32 * d, v[1]);
              }
            }
          }
          // ---- the weights, as fp16 over the scores that have been read
          const float shift = P_BIAS - (mx == -INFINITY ? 0.0f : mx);
          float l[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int b = 0; b < 4; b++) {
            tm_wait_ld(v[b & 1]);
            if (b < 3) tm_ld32(tS + 32 * (b + 1), v[(b + 1) & 1]);
            if (masked) {
              const uint32_t ok = seen(b);
#pragma unroll
              for (int e = 0; e < 32; e++)
                if (!((ok >> e) & 1u)) v[b & 1][e] = __float_as_uint(hidden);
            }
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float p0 = exp2_fast(fmaf(__uint_as_float(v[b & 1][e]), a.scale_log2, shift));
              const float p1 = exp2_fast(fmaf(__uint_as_float(v[b & 1][e + 1]), a.scale_log2, shift));
              l[(e >> 1) & 3] += p0 + p1;
              pk[e >> 1] = pack_f16(p0, p1);
            }
            tm_st16(tS + 16 * b, pk);  // columns of scores 16 b .. 16 b + 15, read at b / 2
          }
          sum += (l[0] + l[1]) + (l[2] + l[3]);
          tm_wait_st();
          if (masked) {
            const uint32_t item = item0 + item_v(i, n), slot = item % TC_RING;
            wait(sh.full[slot], item / TC_RING);
            __syncwarp();
            const unsigned long long bad[2] = {sh.bad[slot][0], sh.bad[slot][1]};
            if ((bad[0] | bad[1]) != 0ull) {
              for (int b = 0; b < 2; b++)
                for (unsigned long long left = bad[b]; left != 0ull; left &= left - 1ull) {
                  const int key = 64 * b + __ffsll((long long)left) - 1;
                  const float p = half_of(tm_ld1(tS + (key >> 1)), key & 1);
                  const __half* src = a.v;
                  if (tree) {
                    src = a.v_new + ((int64_t)s * a.nt + key) * a.kv_stride + kvh * HD;
                  } else {
                    const int at = base + key, e = at / a.page_size;
                    src += (((int64_t)a.table[(int64_t)q.slot * a.max_pages + e] * a.nkv + kvh) * a.page_size +
                            (at - e * a.page_size)) * HD;
                  }
                  for (int d = 0; d < CH; d++) {
                    tm_ld32(tO + 32 * d, v[0]);
                    tm_wait_ld(v[0]);
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                      const uint4 vv = *reinterpret_cast<const uint4*>(src + 32 * d + 8 * x);
                      if (p > 0.0f && odd_chunk(vv)) {
                        const uint32_t ww[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                        for (int e = 0; e < 8; e++)
                          v[0][8 * x + e] = __float_as_uint(fmaf(p, half_of(ww[e >> 1], e & 1), __uint_as_float(v[0][8 * x + e])));
                      }
                    }
                    __syncwarp();
                    tm_st32(tO + 32 * d, v[0]);
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
      const size_t slot = (size_t)blockIdx.x * 2 + (w > w0 ? 1 : 0);
      const int hd0 = kvh * a.G + (live ? m % a.G : 0);
      __half* dst = a.out + (((int64_t)s * a.nt + node) * a.nq + hd0) * HD;
      float* po = a.part_o + (slot * ROWS + (TWO ? 128 * j : 0) + r) * HD;
      // 32 dimensions of the row, as they are, or times 1 / sum as fp16
      auto put = [&](int d, const uint32_t (&o)[32], float inv) {
        if (!live) return;
        if (whole) {
#pragma unroll
          for (int x = 0; x < 4; x++) {
            uint4 y;
            auto f = [&](int e) { return __uint_as_float(o[8 * x + e]) * inv; };
            y.x = pack_f16(f(0), f(1));
            y.y = pack_f16(f(2), f(3));
            y.z = pack_f16(f(4), f(5));
            y.w = pack_f16(f(6), f(7));
            *reinterpret_cast<uint4*>(dst + 32 * d + 8 * x) = y;
          }
        } else {
#pragma unroll
          for (int x = 0; x < 8; x++)
            *reinterpret_cast<uint4*>(po + 32 * d + 4 * x) =
                make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
      };
      if (TWO) {
        if (warp_live) {
          const float inv = 1.0f / sum;
#pragma unroll
          for (int d = 0; d < CH; d++) {
            uint32_t o[32];
            tm_ld32(tO + 32 * d, o);
            tm_wait_ld(o);
            put(d, o, inv);
          }
          if (live && !whole) a.part_ml[slot * ROWS + 128 * j + r] = make_float2(mx, sum);
        }
      } else {
        // stream 1 hands its share to stream 0 through the second q tile,
        // half of the dimensions at a time: x[dimension][row]
        float* x = reinterpret_cast<float*>(smem + Sh::TILE);
        float w_own = 1.0f, w_other = 0.0f;
        if (j == 1) sh.x_ml[r] = make_float2(mx, sum);
#pragma unroll
        for (int half = 0; half < 2; half++) {
          if (n > 1) {
            if (half == 1) asm volatile("bar.sync 3, 256;" ::: "memory");  // the first half has been read
            if (j == 1 && warp_live) {
#pragma unroll
              for (int d = 0; d < CH / 2; d++) {
                uint32_t o[32];
                tm_ld32(tO + 32 * (half * (CH / 2) + d), o);
                tm_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; e++) x[(32 * d + e) * 128 + r] = __uint_as_float(o[e]);
              }
            }
            asm volatile("bar.sync 3, 256;" ::: "memory");
          }
          if (j == 0 && warp_live) {
            if (half == 0) {
              const float2 other = n > 1 ? sh.x_ml[r] : make_float2(-INFINITY, 0.0f);
              const float m2 = fmaxf(mx, other.x), ref = m2 == -INFINITY ? 0.0f : m2;
              w_own = exp2_fast(mx - ref);
              w_other = exp2_fast(other.x - ref);
              sum = sum * w_own + other.y * w_other;
              mx = m2;
              if (live && !whole) a.part_ml[slot * ROWS + r] = make_float2(mx, sum);
            }
            const float inv = 1.0f / sum;
#pragma unroll
            for (int d = 0; d < CH / 2; d++) {
              uint32_t o[32];
              tm_ld32(tO + 32 * (half * (CH / 2) + d), o);
              tm_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; e++) {
                float y = __uint_as_float(o[e]) * w_own;
                if (n > 1) y = fmaf(x[(32 * d + e) * 128 + r], w_other, y);
                o[e] = __float_as_uint(y);
              }
              put(half * (CH / 2) + d, o, inv);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(bar(sh.q_empty));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == ALLOC_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  if (tid == 0) a.part_err[blockIdx.x] = sh.abort != 0 ? 1u : 0u;
}

template <int HD, bool TWO>
cudaError_t launch(const TreeArgs& a, int n_cta, cudaStream_t st) {
  tree_attn_tc_kernel<HD, TWO><<<n_cta, TC_THREADS, tc_smem<HD>(), st>>>(a);
  return cudaGetLastError();
}

template <int HD, bool TWO>
void init() {
  cudaFuncSetAttribute(tree_attn_tc_kernel<HD, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)tc_smem<HD>());
}

}  // namespace

cudaError_t tree_tc_launch(const TreeArgs& a, int hd, int n_cta, cudaStream_t st) {
  if (hd == 128) return a.rows == 256 ? launch<128, true>(a, n_cta, st) : launch<128, false>(a, n_cta, st);
  return a.rows == 256 ? launch<64, true>(a, n_cta, st) : launch<64, false>(a, n_cta, st);
}

void tree_tc_init_attrs() {
  init<64, false>();
  init<64, true>();
  init<128, false>();
  init<128, true>();
}
