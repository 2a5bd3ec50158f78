// blocks.cu -- which blocks of a cache a query attends to: digests of the
// blocks (spec_block_digest), scores from them (spec_block_scores), and the
// selection of the largest (spec_block_select).
#include <climits>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "key_warp.cuh"

namespace {

// ---------------------------------------------------------------------------
// digests: a warp per block, 16 bytes a lane and load, several rows of the block a
// load; the lanes that hold the same channels are joined at the end
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

template <int HD, bool Q4>
__global__ void __launch_bounds__(DG_THREADS)
digest_kernel(const spec_digest dg, const Keys keys, int n, const int32_t* __restrict__ slots,
              const int32_t* __restrict__ pos0, int split, int32_t* __restrict__ status) {
  constexpr int ROW = Q4 ? HD / 2 : HD * 2, LANES = ROW / 16, PER = 32 / LANES;  // bytes; lanes and rows of a load
  constexpr int REGS = Q4 ? 16 : 4, U = Q4 ? 4 : 8;
  grid_dep_begin();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * DG_WARPS + (threadIdx.x >> 5);
  const int y = (int)(w % split);
  const long long unit = w / split;
  const int h = (int)(unit % dg.n_kv_heads), layer = (int)(unit / dg.n_kv_heads % dg.n_layers);
  const long long i_ = unit / dg.n_kv_heads / dg.n_layers;
  if (i_ >= n) return;
  const int i = (int)i_, slot = slots[i], p0 = pos0 != nullptr ? pos0[i] : 0;
  int st = 0, len = 0;
  if (slot < 0 || slot >= dg.n_slots)
    st |= SPEC_ST_SLOT;
  else
    len = dg.len[slot];
  if (p0 < 0 || len < 0 || len > dg.max_pages * dg.page_size) st |= SPEC_ST_FULL;
  const int block = dg.block, per = dg.page_size / block, nb = st == 0 ? (int)(((int64_t)len + block - 1) / block) : 0;
  const int32_t* row = dg.table + (int64_t)(st == 0 ? slot : 0) * dg.max_pages;
  if (h == 0 && layer == 0 && y == 0) {  // the entry's status
    bool bad = false;
    if (p0 / block < nb)
      for (int e = p0 / block / per + lane; e <= (nb - 1) / per; e += 32) bad |= row[e] < 0 || row[e] >= dg.n_pages;
    if (__any_sync(0xffffffffu, bad)) st |= SPEC_ST_PAGE;
    if (lane == 0) status[i] = st;
  }
  for (int64_t b = (int64_t)p0 / block + y; b < nb; b += split) {
    const int pg = row[b / per];
    if (pg < 0 || pg >= dg.n_pages) continue;
    const int64_t head = (int64_t)pg * dg.n_kv_heads + h;
    const int64_t r0 = (int64_t)layer * keys.layer_stride + head * dg.page_size + (b % per) * block;
    const int rows = (int)min((int64_t)block, len - b * block);
    uint32_t lo[REGS], hi[REGS];
#pragma unroll
    for (int x = 0; x < REGS; x++) {
      lo[x] = 0x7C007C00u;
      hi[x] = 0xFC00FC00u;
    }
    const uint8_t* src = keys.rows + r0 * ROW + (lane % LANES) * 16;
    const __half* sc = Q4 ? keys.scales + r0 * (HD / 32) + lane % LANES : nullptr;
    for (int r = lane / LANES; r < rows; r += PER * U) {
      uint4 v[U];
      uint32_t s[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int at = min(r + u * PER, rows - 1);  // (a row again changes nothing)
        v[u] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)at * ROW));
        if (Q4) s[u] = __half_as_ushort(__ldg(sc + (int64_t)at * (HD / 32))) * 0x10001u;
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        const uint32_t q[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int x = 0; x < REGS; x++) {
          // codes: word x / 4; elements 0, 2 | 1, 3 | 16, 18 | 17, 19 of its four
          const uint32_t val = !Q4 ? q[x % 4]
                                   : kw_hmul2(x & 2 ? q4_high(q[x / 4] >> (x & 1 ? 8 : 0))
                                                    : q4_low(q[x / 4] >> (x & 1 ? 8 : 0)), s[u]);
          lo[x] = min2(lo[x], val);
          hi[x] = max2(hi[x], val);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < REGS; x++)
#pragma unroll
      for (int off = LANES; off < 32; off <<= 1) {
        lo[x] = min2(lo[x], __shfl_xor_sync(0xffffffffu, lo[x], off));
        hi[x] = max2(hi[x], __shfl_xor_sync(0xffffffffu, hi[x], off));
      }
    uint16_t* to = dg.data + (int64_t)layer * dg.layer_stride + (head * per + b % per) * (2 * HD);
    if (lane < LANES) {
      uint4* d[2] = {reinterpret_cast<uint4*>(to), reinterpret_cast<uint4*>(to + HD)};
#pragma unroll
      for (int which = 0; which < 2; which++) {
        const uint32_t(&z)[REGS] = which ? hi : lo;
        if (!Q4) {
          d[which][lane] = make_uint4(z[0], z[1], z[2], z[3]);
        } else {
#pragma unroll
          for (int half = 0; half < 2; half++)
#pragma unroll
            for (int p = 0; p < 2; p++) {  // elements 16 half + 8 p ...: words 2 p, 2 p + 1
              uint32_t e[4];
#pragma unroll
              for (int x = 0; x < 2; x++) {
                const uint32_t even = z[4 * (2 * p + x) + 2 * half], odd = z[4 * (2 * p + x) + 2 * half + 1];
                e[2 * x] = __byte_perm(even, odd, 0x5410);
                e[2 * x + 1] = __byte_perm(even, odd, 0x7632);
              }
              d[which][4 * lane + 2 * half + p] = make_uint4(e[0], e[1], e[2], e[3]);
            }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// scores: sum_d max(q lo, q hi) = min(q, 0) . lo + max(q, 0) . hi, a product over 2 hd
// channels with the digest as it lies in memory: a tile of 16 blocks a warp
// (its digests straight into the A fragments, whose order of channels the queries
// follow), 8 query rows a product, and the maximum over the group's heads
// through shared memory
// ---------------------------------------------------------------------------
constexpr int SC_THREADS = 128, SC_WARPS = 4, SC_ROWS = 64;

struct ScoreArgs {
  spec_digest dg;
  int layer, n_seq, nt, nq, G;
  const int32_t* slots;
  const int32_t* n_nodes;
  const __half* q;
  int64_t q_stride;
  float* scores;
  int64_t ld;
  int32_t* status;
  int nodes, groups;  // nodes of a CTA, CTAs for a sequence's nodes
  int chunks;         // CTAs for a sequence's blocks
};

template <int HD>
__host__ __device__ constexpr int score_q_bytes(int tiles) {
  return tiles * (2 * HD / 16) * 32 * 8;
}

template <int HD>
__global__ void __launch_bounds__(SC_THREADS) scores_kernel(const ScoreArgs a) {
  constexpr int STEPS = 2 * HD / 16, LOADS = 2 * HD / 32;  // 16-byte loads of a lane and row
  extern __shared__ __align__(16) unsigned char smem[];
  grid_dep_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const spec_digest& dg = a.dg;
  const int chunk = blockIdx.x % a.chunks, grp = blockIdx.x / a.chunks % a.groups;
  const int h = blockIdx.x / a.chunks / a.groups % dg.n_kv_heads, s = blockIdx.x / a.chunks / a.groups / dg.n_kv_heads;
  const int slot = a.slots[s], m = a.n_nodes != nullptr ? a.n_nodes[s] : a.nt;
  int st = 0, len = 0;
  if (slot < 0 || slot >= dg.n_slots)
    st |= SPEC_ST_SLOT;
  else
    len = dg.len[slot];
  if (m < 0 || m > a.nt) st |= SPEC_ST_TREE;
  const int block = dg.block, per = dg.page_size / block;
  const int64_t nb = ((int64_t)max(len, 0) + block - 1) / block;
  if (len < 0 || len > dg.max_pages * dg.page_size || nb > a.ld) st |= SPEC_ST_FULL;
  const int32_t* row = dg.table + (int64_t)(st == 0 ? slot : 0) * dg.max_pages;
  if (chunk == 0 && grp == 0 && h == 0) {
    bool bad = false;
    if (st == 0)
      for (int64_t e = tid; e * per < nb; e += SC_THREADS) bad |= row[e] < 0 || row[e] >= dg.n_pages;
    if (__syncthreads_or(bad)) st |= SPEC_ST_PAGE;
    if (tid == 0) a.status[s] = st;
    st &= ~SPEC_ST_PAGE;
  }
  const int node0 = grp * a.nodes, nodes = min(a.nodes, m - node0), rows = nodes * a.G;
  if (st != 0 || nodes <= 0 || (int64_t)chunk * 16 * SC_WARPS >= nb) return;
  const int tiles = (rows + 7) / 8;
  const uint32_t qs = kw_smem(smem);
  for (int e = tid; e < tiles * STEPS * 32; e += SC_THREADS) {
    const int el = e & 31, step = e / 32 % STEPS, n = e / 32 / STEPS;
    const int r = 8 * n + (el >> 2), c = 8 * (4 * (step >> 1) + (el & 3)) + 4 * (step & 1);  // of 2 hd channels
    uint32_t b0 = 0u, b1 = 0u;
    if (r < rows) {
      const int node = node0 + r / a.G, head = h * a.G + r % a.G;
      const uint2 v =
          *reinterpret_cast<const uint2*>(a.q + ((int64_t)s * a.nt + node) * a.q_stride + head * HD + c % HD);
      b0 = c < HD ? min2(v.x, 0u) : max2(v.x, 0u);
      b1 = c < HD ? min2(v.y, 0u) : max2(v.y, 0u);
    }
    kw_sts64(qs + e * 8, b0, b1);
  }
  __syncthreads();
  // [block of the tile][row], a row more to keep the banks apart
  float* x = reinterpret_cast<float*>(smem + score_q_bytes<HD>((a.nodes * a.G + 7) / 8)) + warp * 16 * (SC_ROWS + 1);
  for (int64_t b0 = ((int64_t)chunk * SC_WARPS + warp) * 16; b0 < nb; b0 += (int64_t)a.chunks * SC_WARPS * 16) {
    uint4 v[2][LOADS];
    bool there[2];
#pragma unroll
    for (int half = 0; half < 2; half++) {
      const int64_t b = b0 + 8 * half + g;
      const int pg = b < nb ? row[b / per] : -1;
      there[half] = pg >= 0 && pg < dg.n_pages;
      const uint4* src = reinterpret_cast<const uint4*>(
          dg.data + (int64_t)a.layer * dg.layer_stride +
          (((int64_t)(there[half] ? pg : 0) * dg.n_kv_heads + h) * per + (there[half] ? b % per : 0)) * (2 * HD));
#pragma unroll
      for (int i = 0; i < LOADS; i++) v[half][i] = __ldg(src + 4 * i + t);
    }
    for (int n = 0; n < tiles; n++) {
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < LOADS; i++) {
        const uint2 q0 = kw_lds64(qs + ((n * STEPS + 2 * i) * 32 + lane) * 8);
        const uint2 q1 = kw_lds64(qs + ((n * STEPS + 2 * i + 1) * 32 + lane) * 8);
        const uint32_t a0[4] = {v[0][i].x, v[1][i].x, v[0][i].y, v[1][i].y};
        const uint32_t a1[4] = {v[0][i].z, v[1][i].z, v[0][i].w, v[1][i].w};
        mma_16816(acc, a0, q0.x, q0.y);
        mma_16816(acc, a1, q1.x, q1.y);
      }
#pragma unroll
      for (int e = 0; e < 4; e++)
        x[(g + 8 * (e >> 1)) * (SC_ROWS + 1) + 8 * n + 2 * t + (e & 1)] = there[e >> 1] ? acc[e] : -INFINITY;
    }
    __syncwarp();
    const int64_t b = b0 + (lane & 15);
    for (int i = lane >> 4; i < nodes; i += 2) {
      const float* p = x + (lane & 15) * (SC_ROWS + 1) + i * a.G;
      float top = p[0];
      bool nan = top != top;
      for (int k = 1; k < a.G; k++) {
        nan |= p[k] != p[k];
        top = fmaxf(top, p[k]);
      }
      if (nan) top = __int_as_float(0x7FFFFFFF);
      if (b < nb) a.scores[(((int64_t)s * a.nt + node0 + i) * dg.n_kv_heads + h) * a.ld + b] = top;
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// selection: a CTA per row.  The k-th largest score's bits are found from the
// highest on, by counting the scores that reach each candidate (they stay in
// registers, PER a thread); the rows end early once exactly k scores do.
// ---------------------------------------------------------------------------
struct SelectArgs {
  const int32_t* len;
  int n_slots, block, n_seq, nt, nkv;
  const int32_t* slots;
  const int32_t* n_nodes;
  const float* scores;
  int64_t ld;
  int keep, first, last;
  int32_t* blocks;
  int32_t* status;
};

template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) select_kernel(const SelectArgs a) {
  __shared__ int s_warp[2][THREADS / 32];
  grid_dep_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x;
  const int h = (int)(r % a.nkv), node = (int)(r / a.nkv % a.nt), s = (int)(r / a.nkv / a.nt);
  const int slot = a.slots[s], m = a.n_nodes != nullptr ? a.n_nodes[s] : a.nt;
  int st = 0, len = 0;
  if (slot < 0 || slot >= a.n_slots)
    st |= SPEC_ST_SLOT;
  else
    len = a.len[slot];
  if (m < 0 || m > a.nt) st |= SPEC_ST_TREE;
  const int nb = (int)(((int64_t)max(len, 0) + a.block - 1) / a.block);
  if (len < 0 || nb > a.ld) st |= SPEC_ST_FULL;
  if (h == 0 && node == 0 && tid == 0) a.status[s] = st;
  int32_t* out = a.blocks + r * a.keep;
  if ((st & SPEC_ST_TREE) == 0 && node >= m) return;
  const int k = st != 0 ? 0 : min(nb, a.keep);
  for (int j = k + tid; j < a.keep; j += THREADS) out[j] = -1;
  if (k == nb || st != 0) {
    for (int j = tid; j < k; j += THREADS) out[j] = j;
    return;
  }
  const float* x = a.scores + r * a.ld;
  auto key_of = [&](int j) -> uint32_t {
    if (j >= nb) return 0u;
    if (j < a.first || j >= nb - a.last) return 0xFFFFFFFFu;
    const float f = x[j];
    return f != f ? 0xFF800000u : logit_key(f);
  };
  // this thread's scores: PER neighbours, chunk after chunk of THREADS * PER
  uint32_t key[PER];
  const bool one = nb <= THREADS * PER;
#pragma unroll
  for (int i = 0; i < PER; i++) key[i] = one ? key_of(tid * PER + i) : 0u;
  int which = 0;
  auto count = [&](uint32_t t) {
    int c = 0;
    if (one) {
#pragma unroll
      for (int i = 0; i < PER; i++) c += key[i] >= t;
    } else {
      for (int j = tid; j < nb; j += THREADS) c += key_of(j) >= t;
    }
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) s_warp[which][warp] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; w++) c += s_warp[which][w];
    which ^= 1;
    return c;
  };
  uint32_t t = 0u;
  int reach = nb;
  for (uint32_t bit = 0x80000000u; bit != 0u && reach != k; bit >>= 1) {
    const int c = count(t | bit);
    if (c >= k) {
      t |= bit;
      reach = c;
    }
  }
  // where more reach it than there is room for, they end in equal scores: the
  // lowest blocks of these
  const int over = reach - k;  // equal ones that stay out, the last ones
  const int equal_in = over == 0 ? INT_MAX : (count(t) - count(t + 1u)) - over;
  // (t is no forced block's key: of those there are at most k)
  int base_gt = 0, base_eq = 0;
  for (int c0 = 0; c0 < nb; c0 += THREADS * PER) {
    int gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      if (!one) key[i] = key_of(c0 + tid * PER + i);
      const bool in = key[i] >= t && c0 + tid * PER + i < nb;
      eq += in && over > 0 && key[i] == t;
      gt += in && !(over > 0 && key[i] == t);
    }
    // exclusive sums over the CTA
    int g0 = gt, e0 = eq;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int yg = __shfl_up_sync(0xffffffffu, g0, off), ye = __shfl_up_sync(0xffffffffu, e0, off);
      if (lane >= off) {
        g0 += yg;
        e0 += ye;
      }
    }
    __syncthreads();
    if (lane == 31) {
      s_warp[0][warp] = g0;
      s_warp[1][warp] = e0;
    }
    __syncthreads();
    int all_g = 0, all_e = 0;
    g0 += base_gt - gt;
    e0 += base_eq - eq;
#pragma unroll
    for (int w = 0; w < THREADS / 32; w++) {
      if (w < warp) {
        g0 += s_warp[0][w];
        e0 += s_warp[1][w];
      }
      all_g += s_warp[0][w];
      all_e += s_warp[1][w];
    }
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int j = c0 + tid * PER + i;
      if (key[i] < t || j >= nb) continue;
      const bool tie = over > 0 && key[i] == t;
      if (!tie || e0 < equal_in) out[g0 + min(e0, equal_in)] = j;
      if (tie)
        e0++;
      else
        g0++;
    }
    base_gt += all_g;
    base_eq += all_e;
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
  if (units > INT32_MAX) return fail(SPEC_E_SHAPE, "n * n_layers * n_kv_heads too large");
  // warps of a unit: as many as keep the SMs full, when the blocks are many
  const int64_t most = (int64_t)dg->max_pages * (dg->page_size / dg->block);
  const int split = (int)std::max<int64_t>(1, std::min<int64_t>(most, (int64_t)(device_sms() * 48 / units)));
  const size_t grid = (size_t)((units * split + DG_WARPS - 1) / DG_WARPS);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto kernel = dg->head_dim == 128 ? (q4 ? digest_kernel<128, true> : digest_kernel<128, false>)
                                    : (q4 ? digest_kernel<64, true> : digest_kernel<64, false>);
  const cudaError_t e = launch_dependent(kernel, grid, DG_THREADS, 0, st, *dg, keys, n, slots, pos0, split, status);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("block digest: ") + cudaGetErrorString(e));
  return SPEC_OK;
}

}  // namespace

bool block_fits(int block, int page_size) {
  return (block == 16 || block == 32 || block == 64 || block == 128) && page_size % block == 0;
}

void blocks_init_attrs() {
  const int most = SC_WARPS * 16 * (SC_ROWS + 1) * 4;
  cudaFuncSetAttribute(scores_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       score_q_bytes<64>(SC_ROWS / 8) + most);
  cudaFuncSetAttribute(scores_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       score_q_bytes<128>(SC_ROWS / 8) + most);
}

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
  a.nodes = std::min(nt, SC_ROWS / a.G);
  a.groups = (nt + a.nodes - 1) / a.nodes;
  // a tile of 16 blocks a warp, until there are CTAs for eight an SM
  const int64_t most = std::min<int64_t>(ld, (int64_t)dg->max_pages * (dg->page_size / dg->block));
  const double units = (double)n_seq * dg->n_kv_heads * a.groups;
  const int64_t fill = std::max<int64_t>(1, (int64_t)(8 * device_sms() / units));
  a.chunks = (int)std::min<int64_t>((most + 16 * SC_WARPS - 1) / (16 * SC_WARPS), fill);
  if (units * a.chunks > INT32_MAX) return fail(SPEC_E_SHAPE, "n_seq * nt * n_kv_heads too large");
  const int tiles = (a.nodes * a.G + 7) / 8;
  const size_t smem = (dg->head_dim == 128 ? score_q_bytes<128>(tiles) : score_q_bytes<64>(tiles)) +
                      SC_WARPS * 16 * (SC_ROWS + 1) * sizeof(float);
  init_attrs_once();
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
  const SelectArgs a = {len, n_slots, block, n_seq, nt, n_kv_heads, slots, n_nodes, scores, ld, n_keep, n_first,
                        n_last, blocks, status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t grid = (size_t)rows;
  const cudaError_t e = ld <= 1024   ? launch_dependent(select_kernel<128, 8>, grid, 128, 0, st, a)
                        : ld <= 4096 ? launch_dependent(select_kernel<256, 16>, grid, 256, 0, st, a)
                                     : launch_dependent(select_kernel<512, 32>, grid, 512, 0, st, a);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("block selection: ") + cudaGetErrorString(e));
  return SPEC_OK;
}
