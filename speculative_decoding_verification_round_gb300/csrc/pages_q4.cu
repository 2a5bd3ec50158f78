// pages_q4.cu -- the pages of a KV cache held in 4 bits: rows quantised into
// it (commit), read back, copied; fork, extend and free are the bookkeeping of
// pages.cu.
//
// Two lanes have a block of 32 elements, lane l of them elements 8 l ... 8 l + 7 and 16 +
// 8 l ...: those that share its eight bytes of codes.  (Eight elements a lane, with
// more exchanges and a word of codes each, take 104 us where this takes 73.)
//
// Measured: two prompts of 4097 rows, 8 layers, 8 heads of 128 (253 MB of fp16, 71 of codes
// and scales): commit 73 us, 4.4 TB/s, 68% of the issue slots: the arithmetic of the
// quantisation; reading back 53.5 us, 6.1 TB/s, reads and writes together.  A head's rows to
// a warp, whose codes are neighbours, 78 and 63 (with 32 rows a CTA in the read 65); more rows
// in flight or stores of 32 bytes: no better.  12 paths of up to 16 nodes in 40 layers: 10.5
// and 6.3 us: the launch, then slot, length, page and a barrier in front of the first row (the
// commit's own rows, which hang on the path alone, are loaded behind that, too).
// 12 pages of 64 positions copied in 40 layers 14.0 us (floor 10.4; fp16 42 and 37); extending 48 branches of
// half a shared page 37 (floor 10.2; fp16 52 and 36): issue slots 70%, a division a word, scales
// two bytes at a time.
#include <algorithm>
#include <climits>

#include "common.cuh"

namespace {

constexpr int PQ_THREADS = 256;

__device__ __forceinline__ float half_of(uint32_t v, int hi) {
  return __half2float(__ushort_as_half((unsigned short)(hi ? v >> 16 : v & 0xFFFFu)));
}

// The scale of a block whose element of the largest magnitude is m (finite):
// eight significant bits, exact in fp16, at most 8160 (255 * 32: 8 times it is
// fp16's, too).
__device__ __forceinline__ float block_scale(float m) {
  const float d = -0.125f * m;  // exact
  const uint32_t u = __float_as_uint(d);
  // to eight bits, to even (|d| <= 8188: no overflow), then to fp16's grid
  const float r = __uint_as_float((u + 0x7FFFu + ((u >> 16) & 1u)) & 0xFFFF0000u);
  return fminf(fmaxf(__half2float(__float2half_rn(r)), -8160.0f), 8160.0f);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // a NaN stays one
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two floats at a time.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2f(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2f(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2f(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Half a block of 32 elements (see above; low: elements 8 l ..., high: 16 + 8 l ...) to the
// block's scale (fp16 bits) and its codes' bytes 8 l ... 8 l + 7.
//
// x / d is not divided: y = x (1 / d) is within a few units of it, and one step
// y + (x - y d) (1 / d) then is exact wherever x / d is a half of an odd number.
// Nothing else is near one: x has 11 bits and d 8, so that |x / d - (k + 1/2)| is 0
// or at least 2^-13.  |x / d| is at most 8 (1 + 2^-8) unless d is subnormal in fp16, so
// that only 8 has to be kept from the codes: by a saturated (q + 9) / 16.
struct Half {
  uint32_t scale;
  uint2 codes;
};
__device__ __forceinline__ Half quantise(const uint4& low, const uint4& high) {
  const uint32_t x[8] = {low.x, low.y, low.z, low.w, high.x, high.y, high.z, high.w};
  uint32_t hi = max2(max2(max2(x[0], x[1]), max2(x[2], x[3])), max2(max2(x[4], x[5]), max2(x[6], x[7])));
  uint32_t lo = min2(min2(min2(x[0], x[1]), min2(x[2], x[3])), min2(min2(x[4], x[5]), min2(x[6], x[7])));
  // (the largest, minus the least)
  uint32_t both = max2(__byte_perm(hi, lo, 0x5410) ^ 0x80000000u, __byte_perm(hi, lo, 0x7632) ^ 0x80000000u);
  both = max2(both, __shfl_xor_sync(0xffffffffu, both, 1));
  const float up = half_of(both, 0), down = half_of(both, 1);
  float m = up > down ? up : -down;
  if (__any_sync(0xffffffffu, up == down && up != 0.0f)) {  // the first of both decides
    int first = 128;
    const uint32_t top = both & 0x7FFFu;
#pragma unroll
    for (int e = 15; e >= 0; e--) {
      const uint32_t v = x[e >> 1] >> (16 * (e & 1));
      if ((v & 0x7FFFu) == top) first = 2 * ((e >> 3) * 16 + 8 * (int)(threadIdx.x & 1) + (e & 7)) + (int)(v >> 15 & 1u);
    }
    first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
    if (up == down) m = first & 1 ? -up : up;
  }
  Half out;
  const bool fine = up < INFINITY && down < INFINITY;  // (a NaN is not)
  const float d = fine ? block_scale(m) : 0.0f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  if (d == 0.0f) inv = 0.0f;
  const bool small = __any_sync(0xffffffffu, fabsf(d) < 0x1p-13f);
  out.scale = fine ? __half_as_ushort(__float2half_rn(d + 0.0f)) : 0x7E00u;  // (-0 to 0)
  const uint64_t inv2 = pair_of(inv, inv), neg2 = pair_of(-d, -d), magic = pair_of(12582912.0f, 12582912.0f),
                 back = pair_of(-12582912.0f, -12582912.0f);
  uint32_t u[8];
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const uint64_t f = pair_of(half_of(x[e], 0), half_of(x[e], 1));
    uint64_t y = mul2f(f, inv2);
    y = fma2f(fma2f(y, neg2, f), inv2, y);
    y = add2f(add2f(y, magic), back);  // to whole numbers, to even
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(y));
    uint32_t q;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(q) : "f"(b), "f"(a));
    if (small) q = max2(q, 0xC800C800u);  // -8
    asm("fma.rn.sat.f16x2 %0, %1, %2, %3;" : "=r"(q) : "r"(q), "r"(0x2C002C00u), "r"(0x38803880u));
    // 16 (q + 9) / 16 + 1023 = 1024 + code
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(u[e]) : "r"(q), "r"(0x4C004C00u), "r"(0x63FE63FEu));
  }
  out.codes.x = __byte_perm(u[0], u[1], 0x6420) + __byte_perm(u[4], u[5], 0x6420) * 16u;
  out.codes.y = __byte_perm(u[2], u[3], 0x6420) + __byte_perm(u[6], u[7], 0x6420) * 16u;
  if (!fine) out.codes.x = out.codes.y = 0x88888888u;
  return out;
}

// A CTA has up to CQ_ROWS rows (of a node, all heads) of one entry and layer: a
// warp takes 512 neighbouring elements of K or V, half a block a lane, of every row (every
// second, fourth or eighth one where a row is shorter than 2048 elements), so that what a
// lane's place in the row is, is found once; CQ_FLIGHT rows are in flight.
constexpr int CQ_ROWS = 32, CQ_FLIGHT = 2;
constexpr int RQ_THREADS = 128;  // of the read, with 8 or 16 rows

// Where the rows of a CTA lie in the cache (of head 0), in blocks.
template <int ROWS>
struct RowPlace {
  int64_t at[ROWS];
};
template <int THREADS, int ROWS>
__device__ __forceinline__ void place_rows(const spec_pages_q4& kv, int layer, const int32_t* row, int pos0, int r0, int r1,
                                           RowPlace<ROWS>& p) {
  for (int j = r0 + threadIdx.x; j < r1; j += THREADS) {
    const int pos = pos0 + j, e = pos / kv.page_size;  // (below 2^31)
    p.at[j - r0] = ((int64_t)layer * kv.layer_stride + (int64_t)row[e] * kv.n_kv_heads * kv.page_size + pos -
                    e * kv.page_size) * (kv.head_dim / 32);
  }
}
// The work of a CTA: f(which, r, step, e, block, ok): K or V, rows r, r + step, ... (CQ_FLIGHT of
// them, below r1), this lane's first element e of a row (and eight from e + 16 on), and how many
// blocks behind the row's place (of head 0) its block is; `ok` false for lanes past the
// row.  Whole warps.
template <int THREADS, class F>
__device__ __forceinline__ void each_piece(const spec_pages_q4& kv, int r0, int r1, F&& f) {
  const int nb = kv.head_dim / 32, blocks = kv.n_kv_heads * nb, per = (blocks + 15) / 16;
  constexpr int WARPS = THREADS / 32;
  const int lane = threadIdx.x & 31, step = per >= WARPS / 2 ? 1 : WARPS / 2 / per;
  for (int item = threadIdx.x >> 5; item < per * step * 2; item += WARPS) {
    const int part = item >> 1, phase = part / per, b = (part - phase * per) * 16 + (lane >> 1);
    const bool ok = b < blocks;
    const int h = ok ? b / nb : 0, e = ok ? 32 * b + 8 * (lane & 1) : 0;
    const int64_t block = (int64_t)h * kv.page_size * nb + (ok ? b - h * nb : 0);
    for (int r = r0 + phase; r < r1; r += step * CQ_FLIGHT) f(item & 1, r, step, e, block, ok);
  }
}

__global__ void __launch_bounds__(PQ_THREADS, 5)
q4_commit_kernel(const spec_pages_q4 kv, int n, const int32_t* __restrict__ slots, int nt,
                 const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new, int64_t new_layer_stride,
                 const int32_t* __restrict__ path, const int32_t* __restrict__ n_path,
                 int32_t* __restrict__ new_len, int blocks, int32_t* __restrict__ status) {
  __shared__ RowPlace<CQ_ROWS> place;
  __shared__ int s_node[CQ_ROWS];
  // (No early launch of what follows: its waiting CTAs would take the room of the next ones here,
  // 20.4 us for 8 entries' commit and read instead of 16.4; without programmatic
  // launches 20.6.)
  grid_dep_wait();
  const int i = blockIdx.x / (kv.n_layers * blocks);
  const int layer = blockIdx.x / blocks % kv.n_layers, blk = blockIdx.x % blocks;
  const int slot = slots[i], np = n_path[i];
  const int32_t* pth = path != nullptr ? path + (int64_t)i * nt : nullptr;
  int st = 0;
  if (slot < 0 || slot >= kv.n_slots) st |= SPEC_ST_SLOT;
  if (np < 0 || np > nt) st |= SPEC_ST_TREE;
  int len = 0;
  const int32_t* row = nullptr;
  if (st == 0) {
    row = kv.table + (int64_t)slot * kv.max_pages;
    len = kv.len[slot];
    if (len < 0 || (int64_t)len + np > (int64_t)kv.max_pages * kv.page_size) st |= SPEC_ST_FULL;
  }
  int bits = 0;
  for (int j = threadIdx.x; j < n; j += PQ_THREADS)
    if (j != i && slots[j] == slot) bits |= SPEC_ST_SLOT;
  const int r0 = blk * CQ_ROWS, r1 = min(np, r0 + CQ_ROWS);
  if (st == 0 && np > 0) {
    if (pth != nullptr)
      for (int j = threadIdx.x; j < np; j += PQ_THREADS)
        if (pth[j] < 0 || pth[j] >= nt) bits |= SPEC_ST_TREE;
    const int e1 = (int)(((int64_t)len + np - 1) / kv.page_size);
    for (int e = len / kv.page_size + threadIdx.x; e <= e1; e += PQ_THREADS) {
      const int p = row[e];
      if (p < 0 || p >= kv.n_pages)
        bits |= SPEC_ST_PAGE;
      else if (kv.refs != nullptr && kv.refs[p] != 1)
        bits |= SPEC_ST_SHARED;
    }
    place_rows<PQ_THREADS>(kv, layer, row, len, r0, r1, place);
    for (int j = r0 + threadIdx.x; j < r1; j += PQ_THREADS) s_node[j - r0] = pth != nullptr ? pth[j] : j;
  }
  if (__syncthreads_or(bits))
    for (int b = 1; b <= SPEC_ST_TREE; b <<= 1)
      if (__syncthreads_or(bits & b)) st |= b;
  if (layer == 0 && blk == 0 && threadIdx.x == 0) {
    status[i] = st;
    if (st == 0 && new_len != nullptr) new_len[slot] = len + np;
  }
  if (st != 0) return;
  const int node = kv.n_kv_heads * kv.head_dim;
  const int64_t src0 = (int64_t)layer * new_layer_stride + (int64_t)i * nt * node;
  const int l = threadIdx.x & 1;
  constexpr int U = CQ_FLIGHT;
  each_piece<PQ_THREADS>(kv, r0, r1, [&](int which, int r, int step, int e, int64_t block, bool ok) {
    const uint16_t* src = (which ? v_new : k_new) + src0 + e;
    uint4 x[U][2];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int rr = r + u * step;
      x[u][0] = x[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (ok && rr < r1) {
        const uint4* p = reinterpret_cast<const uint4*>(src + (int64_t)s_node[rr - r0] * node);
        x[u][0] = __ldcs(p);
        x[u][1] = __ldcs(p + 2);
      }
    }
    uint2* codes = reinterpret_cast<uint2*>(which ? kv.v_qs : kv.k_qs) + 2 * block + l;
    uint16_t* scales = (which ? kv.v_scales : kv.k_scales) + block;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int rr = r + u * step;
      if (rr >= r1) break;  // (whole warps)
      const Half q = quantise(x[u][0], x[u][1]);
      const int64_t at = place.at[rr - r0];
      if (ok) {
        codes[2 * at] = q.codes;
        if (l == 0) scales[at] = (uint16_t)q.scale;
      }
    }
  });
}

// The lengths advanced in place, after every CTA of the commit has read them.
__global__ void q4_advance_kernel(int n, const int32_t* __restrict__ slots, const int32_t* __restrict__ n_path,
                                  int32_t* len, const int32_t* __restrict__ status) {
  grid_dep_wait();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n && status[i] == 0) len[slots[i]] += n_path[i];
}

// The eight values of 8 bytes of codes' low nibbles, or of their high ones.
template <bool HIGH>
__device__ __forceinline__ uint4 eight_values(uint2 c, uint32_t s) {
  const uint32_t s2 = s * 0x10001u;
  auto two = [&](uint32_t w, uint32_t sel) {
    uint32_t u, r;
    const uint32_t b = __byte_perm(w, w, sel);
    if (HIGH)  // (1024 + 16 u) / 16 - 72
      asm("fma.rn.f16x2 %0, %1, %2, %3;"
          : "=r"(u) : "r"(lop3_and_or(b, 0x00F000F0u, 0x64006400u)), "r"(0x2C002C00u), "r"(0xD480D480u));
    else  // (1024 + u) - 1032
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(u) : "r"(lop3_and_or(b, 0x000F000Fu, 0x64006400u)), "r"(0xE408E408u));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(s2));
    return r;
  };
  return make_uint4(two(c.x, 0x1100), two(c.x, 0x3322), two(c.y, 0x1100), two(c.y, 0x3322));
}

// Rows out of the cache.
template <int ROWS>
__global__ void __launch_bounds__(RQ_THREADS, 12)
q4_read_kernel(const spec_pages_q4 kv, const int32_t* __restrict__ slots, int nt, const int32_t* __restrict__ pos0,
               const int32_t* __restrict__ n_pos, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
               int64_t layer_stride, int blocks, int32_t* __restrict__ status) {
  __shared__ RowPlace<ROWS> place;
  grid_dep_wait();
  const int i = blockIdx.x / (kv.n_layers * blocks);
  const int layer = blockIdx.x / blocks % kv.n_layers, blk = blockIdx.x % blocks;
  const int slot = slots[i], np = n_pos[i], p0 = pos0[i];
  int st = 0;
  if (slot < 0 || slot >= kv.n_slots) st |= SPEC_ST_SLOT;
  if (np < 0 || np > nt) st |= SPEC_ST_TREE;
  if (p0 < 0 || (int64_t)p0 + max(np, 0) > (int64_t)kv.max_pages * kv.page_size) st |= SPEC_ST_FULL;
  const int32_t* row = kv.table + (int64_t)(st == 0 ? slot : 0) * kv.max_pages;
  const int r0 = blk * ROWS, r1 = min(np, r0 + ROWS);
  bool bad = false;
  if (st == 0 && np > 0) {
    const int e1 = (int)(((int64_t)p0 + np - 1) / kv.page_size);
    for (int e = p0 / kv.page_size + threadIdx.x; e <= e1; e += RQ_THREADS) bad |= row[e] < 0 || row[e] >= kv.n_pages;
    place_rows<RQ_THREADS>(kv, layer, row, p0, r0, r1, place);
  }
  if (__syncthreads_or(bad)) st |= SPEC_ST_PAGE;
  if (layer == 0 && blk == 0 && threadIdx.x == 0) status[i] = st;
  if (st != 0) return;
  const int node = kv.n_kv_heads * kv.head_dim;
  const int64_t dst0 = (int64_t)layer * layer_stride + (int64_t)i * nt * node;
  const int l = threadIdx.x & 1;
  constexpr int U = CQ_FLIGHT;
  each_piece<RQ_THREADS>(kv, r0, r1, [&](int which, int r, int step, int e, int64_t block, bool ok) {
    const uint2* codes = reinterpret_cast<const uint2*>(which ? kv.v_qs : kv.k_qs) + 2 * block + l;
    const uint16_t* scales = (which ? kv.v_scales : kv.k_scales) + block;
    uint2 c[U];
    uint32_t sc[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int rr = r + u * step;
      const int64_t at = place.at[(rr < r1 ? rr : r) - r0];
      c[u] = __ldg(codes + 2 * at);
      sc[u] = __ldg(scales + at);
    }
    uint16_t* dst = (which ? v : k) + dst0 + e;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int rr = r + u * step;
      if (!ok || rr >= r1) break;
      uint4* p = reinterpret_cast<uint4*>(dst + (int64_t)rr * node);
      __stcs(p, eight_values<false>(c[u], sc[u]));
      __stcs(p + 2, eight_values<true>(c[u], sc[u]));
    }
  });
}

// ---------------------------------------------------------------------------
// copies of pages: the four planes of the first positions of a page
// ---------------------------------------------------------------------------
// Units [e0, e1) of plane `which` of one layer: a head's positions are `unit`
// bytes each (codes: head_dim / 2, scales: head_dim / 16), moved WORD bytes at a
// time.
template <class WORD>
__device__ __forceinline__ void copy_plane(const uint8_t* s, uint8_t* d, uint32_t head, uint32_t run, uint32_t e0,
                                           uint32_t e1) {
  constexpr int U = 8;
  const WORD* src = reinterpret_cast<const WORD*>(s);
  WORD* dst = reinterpret_cast<WORD*>(d);
  const bool whole = run == head;
  for (uint32_t b = e0 + threadIdx.x; b < e1; b += PQ_THREADS * U) {
    WORD t[U];
    uint32_t at[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t e = b + u * PQ_THREADS;
      at[u] = whole ? e : e / run * head + e % run;
      if (e < e1) t[u] = __ldcs(src + at[u]);
    }
#pragma unroll
    for (int u = 0; u < U; u++)
      if (b + u * PQ_THREADS < e1) __stcs(dst + at[u], t[u]);
  }
}

constexpr uint32_t CPQ_WORDS = 8192;  // words of one CTA

// Part `part` of the copy of one page: (layer, K or V, codes or scales' words).
struct CopyShape {
  int code_blocks, scale_blocks;  // CTAs of a plane of a whole page
  __host__ __device__ int per_layer() const { return 2 * (code_blocks + scale_blocks); }
};
__host__ __device__ inline CopyShape copy_shape(int nkv, int page, int hd) {
  const int64_t rows = (int64_t)nkv * page;
  CopyShape c;
  c.code_blocks = (int)((rows * (hd / 32) + CPQ_WORDS - 1) / CPQ_WORDS);   // 16 bytes a word
  c.scale_blocks = (int)((rows * (hd / 32) + CPQ_WORDS - 1) / CPQ_WORDS);  // 2 bytes a word
  return c;
}
__device__ __forceinline__ void copy_part(const spec_pages_q4& kv, const CopyShape& c, int part, int src, int dst,
                                          int n_pos) {
  const int layer = part / c.per_layer(), x = part % c.per_layer();
  const int which = x / (c.code_blocks + c.scale_blocks), y = x % (c.code_blocks + c.scale_blocks);
  const int nb = kv.head_dim / 32;
  const int64_t page = (int64_t)kv.n_kv_heads * kv.page_size * nb, base = (int64_t)layer * kv.layer_stride * nb;
  const uint32_t head = kv.page_size * nb, run = n_pos * nb, words = run * kv.n_kv_heads;
  if (y < c.code_blocks) {
    uint8_t* p = which ? kv.v_qs : kv.k_qs;
    const uint32_t e0 = y * CPQ_WORDS;
    copy_plane<uint4>(p + (base + src * page) * 16, p + (base + dst * page) * 16, head, run, e0,
                      min(words, e0 + CPQ_WORDS));
  } else {
    uint8_t* p = reinterpret_cast<uint8_t*>(which ? kv.v_scales : kv.k_scales);
    const uint32_t e0 = (y - c.code_blocks) * CPQ_WORDS;
    copy_plane<unsigned short>(p + (base + src * page) * 2, p + (base + dst * page) * 2, head, run, e0,
                               min(words, e0 + CPQ_WORDS));
  }
}

__global__ void __launch_bounds__(PQ_THREADS)
q4_copy_kernel(const spec_pages_q4 kv, int n, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
               const int32_t* __restrict__ n_pos, const CopyShape c, int32_t* __restrict__ status) {
  const int per = kv.n_layers * c.per_layer();
  const int i = blockIdx.x / per, part = blockIdx.x % per;
  const int a = src[i], b = dst[i];
  const int np = n_pos != nullptr ? n_pos[i] : kv.page_size;
  int st = 0;
  if (a < 0 || a >= kv.n_pages || b < 0 || b >= kv.n_pages) st |= SPEC_ST_SLOT;
  if (np < 0 || np > kv.page_size) st |= SPEC_ST_PAGE;
  bool hit = a == b;  // what another entry writes or reads, or reads what one writes
  for (int j = threadIdx.x; j < n; j += PQ_THREADS) {
    const int s = src[j], d = dst[j];
    hit |= (j != i && d == b) || s == b || d == a;
  }
  if (__syncthreads_or(hit)) st |= SPEC_ST_SLOT;
  if (part == 0 && threadIdx.x == 0) status[i] = st;
  if (st == 0 && np > 0) copy_part(kv, c, part, a, b, np);
}

// The filled positions of the pages that an extension has replaced: one CTA per
// (entry, layer, part of the page).
__global__ void __launch_bounds__(PQ_THREADS)
q4_cow_kernel(const spec_pages_q4 kv, const int32_t* __restrict__ slots, const int32_t* __restrict__ copies,
              const CopyShape c) {
  const int per = kv.n_layers * c.per_layer(), i = blockIdx.x / per;
  grid_dep_wait();
  const int a = copies[2 * i], b = copies[2 * i + 1];
  if (a < 0) return;
  copy_part(kv, c, blockIdx.x % per, a, b, kv.len[slots[i]] % kv.page_size);
}

int check_list(const void* a, const void* status, int n) {
  if (a == nullptr || status == nullptr) return fail(SPEC_E_INVALID, "null argument");
  if (n < 1) return fail(SPEC_E_SHAPE, "n >= 1 required");
  return SPEC_OK;
}
int launched(const char* what, cudaError_t e) {
  return e == cudaSuccess ? SPEC_OK : fail(SPEC_E_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
// Rows of fp16 in or out beside the cache.
int check_rows(const spec_pages_q4* kv, int n, int nt, const void* k, const void* v, int64_t* stride) {
  if (k == nullptr || v == nullptr) return fail(SPEC_E_INVALID, "null argument");
  if (nt < 1) return fail(SPEC_E_SHAPE, "nt >= 1 required");
  if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) != 0)
    return fail(SPEC_E_SHAPE, "k and v rows must be 16-byte aligned");
  const double rows = (double)n * nt * kv->n_kv_heads * kv->head_dim;
  if (rows > 4.0e15 || (double)*stride * kv->n_layers > 4.0e15) return fail(SPEC_E_SHAPE, "the rows are too large");
  const int64_t layer = (int64_t)n * nt * kv->n_kv_heads * kv->head_dim;
  if (*stride == 0) *stride = layer;
  if (*stride % 8 != 0 || (kv->n_layers > 1 && *stride < layer))
    return fail(SPEC_E_SHAPE, "the rows' layer stride must be a multiple of 8 and hold a layer's rows");
  if ((double)n * kv->n_layers * ((nt + 7) / 8) > INT32_MAX)
    return fail(SPEC_E_SHAPE, "n * n_layers * nt too large");
  return SPEC_OK;
}

}  // namespace

// The bookkeeping of a cache in 4 bits as spec_pages (k and v are not to be
// read: they stand for the codes).
spec_pages book_of(const spec_pages_q4* kv) {
  spec_pages p;
  p.k = reinterpret_cast<uint16_t*>(kv->k_qs);
  p.v = reinterpret_cast<uint16_t*>(kv->v_qs);
  p.layer_stride = kv->layer_stride * kv->head_dim;
  p.n_layers = kv->n_layers;
  p.n_pages = kv->n_pages;
  p.n_kv_heads = kv->n_kv_heads;
  p.page_size = kv->page_size;
  p.head_dim = kv->head_dim;
  p.n_slots = kv->n_slots;
  p.max_pages = kv->max_pages;
  p.table = kv->table;
  p.refs = kv->refs;
  p.len = kv->len;
  return p;
}

int check_pages_q4(const spec_pages_q4* kv, bool book) {
  if (kv == nullptr || kv->k_qs == nullptr || kv->v_qs == nullptr || kv->k_scales == nullptr || kv->v_scales == nullptr)
    return fail(SPEC_E_INVALID, "null pages or cache");
  if (kv->head_dim < 32 || kv->head_dim % 32 != 0)
    return fail(SPEC_E_SHAPE, "bad page dimensions (head_dim must be a multiple of 32)");
  if (((reinterpret_cast<uintptr_t>(kv->k_qs) | reinterpret_cast<uintptr_t>(kv->v_qs) |
        reinterpret_cast<uintptr_t>(kv->k_scales) | reinterpret_cast<uintptr_t>(kv->v_scales)) & 15u) != 0)
    return fail(SPEC_E_SHAPE, "codes and scales must be 16-byte aligned");
  if (kv->layer_stride < 0 || (double)kv->layer_stride * kv->head_dim > 4.0e15)
    return fail(SPEC_E_SHAPE, "bad layer_stride");
  const spec_pages p = book_of(kv);
  return check_pages(&p, book);
}

extern "C" int spec_pages_q4_copy(const spec_pages_q4* kv, int n, const int32_t* src, const int32_t* dst,
                                  const int32_t* n_pos, int32_t* status, void* stream) {
  int rc = check_pages_q4(kv, false);
  if (rc == SPEC_OK) rc = check_list(src, status, n);
  if (rc == SPEC_OK) rc = check_list(dst, status, n);
  if (rc != SPEC_OK) return rc;
  const CopyShape c = copy_shape(kv->n_kv_heads, kv->page_size, kv->head_dim);
  const double grid = (double)n * kv->n_layers * c.per_layer();
  if (grid > INT32_MAX) return fail(SPEC_E_SHAPE, "n * n_layers * page too large");
  q4_copy_kernel<<<(unsigned)grid, PQ_THREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(*kv, n, src, dst, n_pos, c,
                                                                                          status);
  return launched("4-bit page copy", cudaGetLastError());
}

extern "C" int spec_pages_q4_fork(const spec_pages_q4* kv, int n, const int32_t* src, const int32_t* dst,
                                  int32_t* status, void* stream) {
  const int rc = check_pages_q4(kv, true);
  if (rc != SPEC_OK) return rc;
  const spec_pages p = book_of(kv);
  return spec_pages_fork(&p, n, src, dst, status, stream);
}

extern "C" int spec_pages_q4_free(const spec_pages_q4* kv, int n, const int32_t* slots, int32_t* status,
                                  void* stream) {
  const int rc = check_pages_q4(kv, true);
  if (rc != SPEC_OK) return rc;
  const spec_pages p = book_of(kv);
  return spec_pages_free(&p, n, slots, status, stream);
}

extern "C" int spec_pages_q4_extend(const spec_pages_q4* kv, int n, const int32_t* slots, const int32_t* n_new,
                                    int32_t* copies, int32_t* status, void* stream) {
  int rc = check_pages_q4(kv, true);
  if (rc != SPEC_OK) return rc;
  const spec_pages p = book_of(kv);
  const CopyShape c = copy_shape(kv->n_kv_heads, kv->page_size, kv->head_dim);
  if ((double)std::max(n, 1) * kv->n_layers * c.per_layer() > INT32_MAX)
    return fail(SPEC_E_SHAPE, "n * n_layers * page too large");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = launch_extend_book(&p, n, slots, n_new, copies, status, st);
  if (rc != SPEC_OK) return rc;
  const cudaError_t e = launch_dependent(q4_cow_kernel, (size_t)n * kv->n_layers * c.per_layer(), PQ_THREADS, 0, st,
                                         *kv, slots, (const int32_t*)copies, c);
  return launched("4-bit page extend", e);
}

extern "C" int spec_pages_q4_commit(const spec_pages_q4* kv, int n, const int32_t* slots, int nt,
                                    const uint16_t* k_new, const uint16_t* v_new, int64_t new_layer_stride,
                                    const int32_t* path, const int32_t* n_path, int32_t* new_len, int32_t* status,
                                    void* stream) {
  int rc = check_pages_q4(kv, true);
  if (rc == SPEC_OK) rc = check_list(slots, status, n);
  if (rc == SPEC_OK && n_path == nullptr) rc = fail(SPEC_E_INVALID, "null argument");
  if (rc == SPEC_OK) rc = check_rows(kv, n, nt, k_new, v_new, &new_layer_stride);
  if (rc != SPEC_OK) return rc;
  const int blocks = (nt + CQ_ROWS - 1) / CQ_ROWS;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // lengths written where they are read from go up in a kernel behind
  const uintptr_t a = reinterpret_cast<uintptr_t>(kv->len), b = reinterpret_cast<uintptr_t>(new_len);
  const uintptr_t bytes = (uintptr_t)kv->n_slots * sizeof(int32_t);
  const bool in_place = new_len == nullptr || a == b;
  if (!in_place && a < b + bytes && b < a + bytes)
    return fail(SPEC_E_INVALID, "new_len overlaps len without being len");
  cudaError_t e = launch_dependent(q4_commit_kernel, (size_t)n * kv->n_layers * blocks, PQ_THREADS, 0, st, *kv, n, slots,
                                   nt, k_new, v_new, new_layer_stride, path, n_path, in_place ? nullptr : new_len, blocks,
                                   status);
  if (e == cudaSuccess && in_place)
    e = launch_dependent(q4_advance_kernel, (size_t)(n + 127) / 128, 128, 0, st, n, slots, n_path, kv->len,
                         (const int32_t*)status);
  return launched("4-bit page commit", e);
}

extern "C" int spec_pages_q4_read(const spec_pages_q4* kv, int n, const int32_t* slots, int nt, const int32_t* pos0,
                                  const int32_t* n_pos, uint16_t* k, uint16_t* v, int64_t layer_stride,
                                  int32_t* status, void* stream) {
  int rc = check_pages_q4(kv, true);
  if (rc == SPEC_OK) rc = check_list(slots, status, n);
  if (rc == SPEC_OK && (pos0 == nullptr || n_pos == nullptr)) rc = fail(SPEC_E_INVALID, "null argument");
  if (rc == SPEC_OK) rc = check_rows(kv, n, nt, k, v, &layer_stride);
  if (rc != SPEC_OK) return rc;
  // 8 rows a CTA where CTAs of 16 would be more than are resident (2 prompts of 4097 in 8 layers
  // 53.5 us instead of 57.5, with 32 rows 64; 12 entries of 16 in 40 layers, which are, 7.2 and 6.3)
  const int64_t entries = (int64_t)n * kv->n_layers;
  const bool many = entries * ((nt + 15) / 16) > 12 * (int64_t)device_sms();
  const int rows = many ? 8 : 16, blocks = (nt + rows - 1) / rows;
  return launched("4-bit page read",
                  launch_dependent(many ? q4_read_kernel<8> : q4_read_kernel<16>, (size_t)entries * blocks, RQ_THREADS, 0,
                                   reinterpret_cast<cudaStream_t>(stream), *kv, slots, nt, pos0, n_pos, k, v, layer_stride,
                                   blocks, status));
}
