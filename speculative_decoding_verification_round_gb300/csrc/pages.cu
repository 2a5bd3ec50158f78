// pages.cu -- the pages of a KV cache: copy, fork (sharing), extend (copy on
// write, lowest free pages first), commit of an accepted path, free; and
// greedy acceptance along a tree, which gives the path to commit.
//
// The bookkeeping (table, reference counts, lengths) lives in device memory
// and is the whole state: a page is free when its count is zero, so no free
// list has to be kept, and which pages a call takes is a function of the
// arrays alone.  Every entry of a call is checked by every CTA that works on
// it from arrays that the kernel does not write (or writes only for other
// entries), so an entry is done whole or not at all.
//
// Bound by the bytes moved, or by the launch: 96 pages of 64 positions copied
// in 40 layers (8 heads of 128; 2.01 GB read and written) 296 us, the copy
// bandwidth; 12 prompts of 550 positions freed, forked into four branches each
// and extended by 16 positions, the filled part of 36 last pages copied (0.37
// GB, 55 us of the copy bandwidth) 73 us in four launches; accepted paths of
// 12 x 16 nodes committed in 40 layers (31 MB, 4.6 us) 8.9 us; acceptance
// along one tree 1.9 us, 512 trees of 63 nodes 2.8 us.
#include <climits>

#include "common.cuh"

namespace {

constexpr int PG_THREADS = 256;

// Whether `value` is in list[0, n) at an index other than `skip` (uniform
// over the CTA; every thread calls it).
__device__ __forceinline__ bool listed(const int32_t* __restrict__ list, int n, int value,
                                       int skip) {
  bool hit = false;
  for (int j = threadIdx.x; j < n; j += blockDim.x) hit |= j != skip && list[j] == value;
  return __syncthreads_or(hit);
}

// Whether entry i = (a -> b) writes what another entry writes or reads, or
// reads what one writes.
__device__ __forceinline__ bool clash(const int32_t* __restrict__ src,
                                      const int32_t* __restrict__ dst, int n, int a, int b, int i) {
  bool hit = a == b;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int s = src[j], d = dst[j];
    hit |= (j != i && d == b) || s == b || d == a;
  }
  return __syncthreads_or(hit);
}

// Units [e0, e1) of the first n_pos positions of page `src` (16-byte units, a
// head's positions after another's) to page `dst`, in one of the two caches
// of one layer.  Eight loads in flight a thread; streaming hints, as the data
// is not needed here again and the L2 has better uses.
constexpr int CP_UNITS = 8192;  // of one CTA: 128 KB

__device__ __forceinline__ void copy_page(const spec_pages& kv, int layer, int which, int src,
                                          int dst, int n_pos, uint32_t e0, uint32_t e1) {
  constexpr int U = 8;
  uint16_t* base = (which ? kv.v : kv.k) + (int64_t)layer * kv.layer_stride;
  const uint32_t row16 = kv.head_dim / 8, run = n_pos * row16, head = kv.page_size * row16;
  const int64_t page = (int64_t)head * kv.n_kv_heads;
  const uint4* s = reinterpret_cast<const uint4*>(base) + src * page;
  uint4* d = reinterpret_cast<uint4*>(base) + dst * page;
  const bool whole = run == head;
  for (uint32_t b = e0 + threadIdx.x; b < e1; b += PG_THREADS * U) {
    uint4 t[U];
    uint32_t at[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t e = b + u * PG_THREADS;
      at[u] = whole ? e : e / run * head + e % run;
      if (e < e1) t[u] = __ldcs(s + at[u]);
    }
#pragma unroll
    for (int u = 0; u < U; u++)
      if (b + u * PG_THREADS < e1) __stcs(d + at[u], t[u]);
  }
}

// ---------------------------------------------------------------------------
// copy: one CTA per (entry, layer, K or V, 128 KB of the page)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(PG_THREADS)
pages_copy_kernel(const spec_pages kv, int n, const int32_t* __restrict__ src,
                  const int32_t* __restrict__ dst, const int32_t* __restrict__ n_pos, int blocks,
                  int32_t* __restrict__ status) {
  const int per = 2 * kv.n_layers * blocks;
  const int i = blockIdx.x / per, part = blockIdx.x % per;
  const int a = src[i], b = dst[i];
  const int np = n_pos != nullptr ? n_pos[i] : kv.page_size;
  int st = 0;
  if (a < 0 || a >= kv.n_pages || b < 0 || b >= kv.n_pages) st |= SPEC_ST_SLOT;
  if (np < 0 || np > kv.page_size) st |= SPEC_ST_PAGE;
  if (clash(src, dst, n, a, b, i)) st |= SPEC_ST_SLOT;
  if (part == 0 && threadIdx.x == 0) status[i] = st;
  if (st != 0) return;
  const uint32_t units = (uint32_t)np * (kv.head_dim / 8) * kv.n_kv_heads;
  const uint32_t e0 = (uint32_t)(part % blocks) * CP_UNITS;
  copy_page(kv, part / blocks >> 1, part / blocks & 1, a, b, np, e0, min(units, e0 + CP_UNITS));
}

// ---------------------------------------------------------------------------
// fork: one CTA per entry
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(PG_THREADS)
pages_fork_kernel(const spec_pages kv, int n, const int32_t* __restrict__ src,
                  const int32_t* __restrict__ dst, int32_t* __restrict__ status) {
  const int i = blockIdx.x, a = src[i], b = dst[i];
  int st = 0;
  if (a < 0 || a >= kv.n_slots || b < 0 || b >= kv.n_slots) st |= SPEC_ST_SLOT;
  if (clash(src, dst, n, a, b, i)) st |= SPEC_ST_SLOT;
  if (st == 0) {
    const int32_t* from = kv.table + (int64_t)a * kv.max_pages;
    int32_t* to = kv.table + (int64_t)b * kv.max_pages;
    const int len = kv.len[a];
    const int held = len <= 0 ? 0 : (len - 1) / kv.page_size + 1;
    bool bad = len < 0 || held > kv.max_pages, taken = kv.len[b] != 0;
    for (int j = threadIdx.x; j < kv.max_pages; j += PG_THREADS) {
      taken |= to[j] >= 0;
      if (j < held) bad |= from[j] < 0 || from[j] >= kv.n_pages;
    }
    if (__syncthreads_or(taken)) st |= SPEC_ST_SLOT;
    if (__syncthreads_or(bad)) st |= SPEC_ST_PAGE;
    if (st == 0) {
      for (int j = threadIdx.x; j < held; j += PG_THREADS) {
        const int p = from[j];
        to[j] = p;
        atomicAdd(kv.refs + p, 1);
      }
      if (threadIdx.x == 0) kv.len[b] = len;
    }
  }
  if (threadIdx.x == 0) status[i] = st;
}

// ---------------------------------------------------------------------------
// extend: one CTA does the bookkeeping (an allocation is a prefix sum over
// the entries and a scan of the reference counts for the lowest zeros), then
// a grid copies the replaced pages' filled positions
// ---------------------------------------------------------------------------
constexpr int EX_THREADS = 1024;  // one thread per entry
constexpr int EX_PER = 4;         // reference counts a thread looks at per step

// Inclusive sum over the CTA's threads; *total gets the whole (every thread).
// In 64 bits: each of 1024 entries may want 2^31 pages.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_warp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();  // s_warp of the last call has been read
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return x + (warp > 0 ? s_warp[warp - 1] : 0);
}

__global__ void __launch_bounds__(EX_THREADS)
pages_extend_kernel(const spec_pages kv, int n, const int32_t* __restrict__ slots,
                    const int32_t* __restrict__ n_new, int32_t* __restrict__ copies,
                    int32_t* __restrict__ status) {
  __shared__ int s_slot[EX_THREADS], s_tail[EX_THREADS];
  __shared__ int64_t s_first[EX_THREADS + 1], s_warp[32];
  __shared__ int s_entry[EX_THREADS];  // first table entry that the entry's fresh pages fill
  __shared__ unsigned char s_copy[EX_THREADS];
  const int i = threadIdx.x;
  const bool mine = i < n;
  const int slot = mine ? slots[i] : -1;
  s_slot[i] = slot;
  __syncthreads();
  int st = 0, tail = -1, j0 = 0;
  int64_t need = 0;
  bool partial = false;
  if (mine) {
    if (slot < 0 || slot >= kv.n_slots) st |= SPEC_ST_SLOT;
    for (int j = 0; j < n; j++)
      if (j != i && s_slot[j] == slot) st |= SPEC_ST_SLOT;
    if (st == 0) {
      const int32_t* row = kv.table + (int64_t)slot * kv.max_pages;
      const int len = kv.len[slot], add = n_new[i];
      const int64_t end = (int64_t)len + add;
      const int64_t want = len < 0 || add < 0 ? 0 : (end + kv.page_size - 1) / kv.page_size;
      if (len < 0 || add < 0) {
        st |= SPEC_ST_PAGE;
      } else if (want > kv.max_pages) {
        st |= SPEC_ST_FULL;
      } else {
        const int last = len / kv.page_size;  // the entry of position len
        partial = len % kv.page_size != 0;
        j0 = last;
        if (partial) {
          tail = row[last];
          if (tail < 0 || tail >= kv.n_pages) st |= SPEC_ST_PAGE;
          j0 = last + 1;
        }
        // pages reserved by an earlier call stay; none may be shared, and
        // from the first gap on every entry has to be empty
        while (j0 < want && row[j0] >= 0) {
          if (row[j0] >= kv.n_pages)
            st |= SPEC_ST_PAGE;
          else if (kv.refs[row[j0]] > 1)
            st |= SPEC_ST_SHARED;
          j0++;
        }
        for (int j = j0; j < want; j++)
          if (row[j] >= 0) st |= SPEC_ST_PAGE;
        need = want > j0 ? want - j0 : 0;
        if (add == 0) tail = -1, partial = false;  // nothing will be written
      }
    }
  }
  if (st != 0 || !partial) tail = -1;
  s_tail[i] = tail;
  __syncthreads();
  // a shared tail is copied by each of its holders here but the last one
  // left: entry i copies iff more than one holder remains after the copies
  // of the entries before it
  bool copy = false;
  if (tail >= 0) {
    int before = 0;
    for (int j = 0; j < i; j++) before += s_tail[j] == tail;
    copy = kv.refs[tail] - before > 1;
  }
  if (st != 0) need = 0;
  need += copy;
  int64_t total;
  const int64_t incl = block_scan(need, s_warp, &total);
  s_first[i + 1] = incl;
  if (i == 0) s_first[0] = 0;
  s_entry[i] = j0;
  s_copy[i] = copy;
  __syncthreads();
  // the k-th free page (in page order) belongs to the entry whose range of
  // the prefix sum holds k: first its copy, then its entries j0, j0 + 1, ...
  int64_t found = 0;
  const int64_t most = total <= kv.n_pages ? kv.n_pages : 0;  // (more than the pool has: none is given out)
  for (int64_t base = 0; base < most && found < total; base += EX_THREADS * EX_PER) {
    const int64_t p0 = base + i * EX_PER;
    int free_mask = 0;
#pragma unroll
    for (int u = 0; u < EX_PER; u++)
      if (p0 + u < kv.n_pages && kv.refs[p0 + u] == 0) free_mask |= 1 << u;
    int64_t here;
    const int64_t upto = block_scan(__popc(free_mask), s_warp, &here);
    int64_t k = found + upto - __popc(free_mask);
    for (int m = free_mask; m != 0 && k < total; m &= m - 1, k++) {
      const int p = (int)p0 + __ffs(m) - 1;
      int lo = 0, hi = EX_THREADS - 1;  // the last entry with s_first <= k
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_first[mid] <= k) lo = mid; else hi = mid - 1;
      }
      const int64_t idx = k - s_first[lo];
      if (s_copy[lo] && idx == 0)
        copies[2 * lo + 1] = p;
      else
        kv.table[(int64_t)s_slot[lo] * kv.max_pages + s_entry[lo] + idx - s_copy[lo]] = p;
      kv.refs[p] = 1;
    }
    found += here;
  }
  __syncthreads();
  const bool full = found < total;
  if (mine) {
    int32_t* row = kv.table + (int64_t)slot * kv.max_pages;
    int from = -1, to = -1;
    if (st == 0) {
      if (full) {  // take back what was given out
        st |= SPEC_ST_FULL;
        const int64_t k0 = s_first[i];
        for (int64_t idx = 0; idx < need && k0 + idx < found; idx++) {
          if (copy && idx == 0) {
            kv.refs[copies[2 * i + 1]] = 0;
          } else {
            const int64_t e = s_entry[i] + idx - (copy ? 1 : 0);
            kv.refs[row[e]] = 0;
            row[e] = -1;
          }
        }
      } else if (copy) {
        from = tail;
        to = copies[2 * i + 1];
        row[kv.len[slot] / kv.page_size] = to;
        atomicSub(kv.refs + from, 1);
      }
    }
    copies[2 * i] = from;
    copies[2 * i + 1] = to;
    status[i] = st;
  }
}

// The filled positions of the replaced pages: one CTA per (entry, layer).
__global__ void __launch_bounds__(PG_THREADS)
pages_cow_kernel(const spec_pages kv, const int32_t* __restrict__ slots,
                 const int32_t* __restrict__ copies) {
  const int i = blockIdx.x / kv.n_layers, layer = blockIdx.x % kv.n_layers;
  grid_dep_wait();
  const int a = copies[2 * i], b = copies[2 * i + 1];
  if (a < 0) return;
  const int filled = kv.len[slots[i]] % kv.page_size;
  const uint32_t units = (uint32_t)filled * (kv.head_dim / 8) * kv.n_kv_heads;
  copy_page(kv, layer, 0, a, b, filled, 0, units);
  copy_page(kv, layer, 1, a, b, filled, 0, units);
}

// ---------------------------------------------------------------------------
// commit: one CTA per (entry, layer, block of rows)
// ---------------------------------------------------------------------------
constexpr int CM_ROWS = 64;

__global__ void __launch_bounds__(PG_THREADS)
pages_commit_kernel(const spec_pages kv, int n, const int32_t* __restrict__ slots, int nt,
                    const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new,
                    int64_t new_layer_stride, const int32_t* __restrict__ path,
                    const int32_t* __restrict__ n_path, int32_t* __restrict__ new_len,
                    int blocks, int32_t* __restrict__ status) {
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
  bool dup = false, bad_node = false, bad_page = false, shared = false;
  for (int j = threadIdx.x; j < n; j += PG_THREADS) dup |= j != i && slots[j] == slot;
  if (st == 0 && np > 0) {
    if (pth != nullptr)
      for (int j = threadIdx.x; j < np; j += PG_THREADS) bad_node |= pth[j] < 0 || pth[j] >= nt;
    const int e1 = (int)(((int64_t)len + np - 1) / kv.page_size);
    for (int e = len / kv.page_size + threadIdx.x; e <= e1; e += PG_THREADS) {
      const int p = row[e];
      if (p < 0 || p >= kv.n_pages)
        bad_page = true;
      else if (kv.refs != nullptr && kv.refs[p] != 1)
        shared = true;
    }
  }
  const int bits = (dup ? SPEC_ST_SLOT : 0) | (bad_node ? SPEC_ST_TREE : 0) |
                   (bad_page ? SPEC_ST_PAGE : 0) | (shared ? SPEC_ST_SHARED : 0);
  // the OR over the CTA of four flags
  if (__syncthreads_or(bits)) {
    if (__syncthreads_or(bits & SPEC_ST_SLOT)) st |= SPEC_ST_SLOT;
    if (__syncthreads_or(bits & SPEC_ST_TREE)) st |= SPEC_ST_TREE;
    if (__syncthreads_or(bits & SPEC_ST_PAGE)) st |= SPEC_ST_PAGE;
    if (__syncthreads_or(bits & SPEC_ST_SHARED)) st |= SPEC_ST_SHARED;
  }
  if (layer == 0 && blk == 0 && threadIdx.x == 0) {
    status[i] = st;
    if (st == 0 && new_len != nullptr) new_len[slot] = len + np;
  }
  if (st != 0) return;
  const int row16 = kv.head_dim / 8, node16 = row16 * kv.n_kv_heads;
  const int64_t head = (int64_t)kv.page_size * kv.head_dim;
  const int64_t src0 = (int64_t)layer * new_layer_stride + (int64_t)i * nt * node16 * 8;
  const int64_t dst0 = (int64_t)layer * kv.layer_stride;
  const int r0 = blk * CM_ROWS, r1 = min(np, r0 + CM_ROWS);
  for (int e = threadIdx.x; e < (r1 - r0) * node16; e += PG_THREADS) {
    const int j = r0 + e / node16, w = e % node16, h = w / row16, u = w % row16;
    const int node = pth != nullptr ? pth[j] : j;
    const int64_t pos = (int64_t)len + j;
    const int p = row[pos / kv.page_size], at = (int)(pos % kv.page_size);
    const int64_t so = src0 + ((int64_t)node * node16 + w) * 8;
    const int64_t d = dst0 + ((int64_t)p * kv.n_kv_heads + h) * head + (int64_t)at * kv.head_dim + u * 8;
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(k_new + so));
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(v_new + so));
    *reinterpret_cast<uint4*>(kv.k + d) = a;
    *reinterpret_cast<uint4*>(kv.v + d) = b;
  }
}

// The lengths advanced in place, after every CTA of the commit has read them.
__global__ void pages_advance_kernel(int n, const int32_t* __restrict__ slots,
                                     const int32_t* __restrict__ n_path, int32_t* len,
                                     const int32_t* __restrict__ status) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n && status[i] == 0) len[slots[i]] += n_path[i];
}

// ---------------------------------------------------------------------------
// free: one CTA per entry
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(PG_THREADS)
pages_free_kernel(const spec_pages kv, int n, const int32_t* __restrict__ slots,
                  int32_t* __restrict__ status) {
  const int i = blockIdx.x, slot = slots[i];
  int st = 0;
  if (slot < 0 || slot >= kv.n_slots || listed(slots, n, slot, i)) st |= SPEC_ST_SLOT;
  if (st == 0) {
    int32_t* row = kv.table + (int64_t)slot * kv.max_pages;
    bool bad = false;
    for (int j = threadIdx.x; j < kv.max_pages; j += PG_THREADS) {
      const int p = row[j];
      if (p >= 0 && p < kv.n_pages)
        atomicSub(kv.refs + p, 1);
      else if (p != -1)
        bad = true;
      if (p != -1) row[j] = -1;
    }
    if (__syncthreads_or(bad)) st |= SPEC_ST_PAGE;
    if (threadIdx.x == 0) kv.len[slot] = 0;
  }
  if (threadIdx.x == 0) status[i] = st;
}

// ---------------------------------------------------------------------------
// greedy acceptance along a tree: one warp per sequence, lane l holding nodes
// l and l + 32; a step down is two ballots, and the whole is a chain of
// depth + 1 of them on registers
// ---------------------------------------------------------------------------
constexpr int AT_WARPS = 4;
static_assert(SPEC_MAX_TREE == 64, "two nodes a lane");

__global__ void __launch_bounds__(AT_WARPS * 32)
accept_tree_kernel(const int32_t* __restrict__ argmax, const int32_t* __restrict__ tokens,
                   const int32_t* __restrict__ parents, const int32_t* __restrict__ n_nodes,
                   int n_seq, int nt, int32_t* __restrict__ path, int32_t* __restrict__ n_path,
                   int32_t* __restrict__ emitted) {
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.x * AT_WARPS + (threadIdx.x >> 5);
  if (s >= n_seq) return;  // whole warps
  const int64_t base = (int64_t)s * nt;
  const int m = n_nodes != nullptr ? n_nodes[s] : nt;
  int par[2], tok[2], top[2];
  bool bad = m < 0 || m > nt;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int i = lane + 32 * h;
    par[h] = tok[h] = top[h] = -1;
    if (i < nt) {
      par[h] = parents[base + i];
      tok[h] = tokens[base + i];
      top[h] = argmax[base + i];
    }
    if (i < m) bad |= par[h] < -1 || par[h] >= i || (i == 0 && par[h] != -1);
  }
  bad = __any_sync(0xffffffffu, bad);
  int out_path[2] = {-1, -1}, out_em[2] = {-1, -1}, cnt = 0;
  if (!bad && m > 0) {
    int cur = 0;
    for (;;) {
      const int am = __shfl_sync(0xffffffffu, cur < 32 ? top[0] : top[1], cur & 31);
#pragma unroll
      for (int h = 0; h < 2; h++)
        if (cnt == lane + 32 * h) {
          out_path[h] = cur;
          out_em[h] = am;
        }
      cnt++;
      const unsigned lo = __ballot_sync(0xffffffffu, lane < m && par[0] == cur && tok[0] == am);
      const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < m && par[1] == cur && tok[1] == am);
      if (lo == 0u && hi == 0u) break;
      cur = lo != 0u ? __ffs(lo) - 1 : 31 + __ffs(hi);  // children are numbered above their parent
    }
  }
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int i = lane + 32 * h;
    if (i < nt) {
      path[base + i] = out_path[h];
      emitted[base + i] = out_em[h];
    }
  }
  if (lane == 0) n_path[s] = bad ? -1 : cnt;
}

// 16-byte units of one page of one layer's K (or V): below 2^31 (check_pages).
int64_t page_units(const spec_pages* kv) {
  return (int64_t)kv->n_kv_heads * kv->page_size * (kv->head_dim / 8);
}

int check_list(const void* a, const void* status, int n) {
  if (a == nullptr || status == nullptr) return fail(SPEC_E_INVALID, "null argument");
  if (n < 1) return fail(SPEC_E_SHAPE, "n >= 1 required");
  return SPEC_OK;
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : fail(SPEC_E_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

}  // namespace

int check_pages(const spec_pages* kv, bool book) {
  if (kv == nullptr || kv->k == nullptr || kv->v == nullptr)
    return fail(SPEC_E_INVALID, "null pages or cache");
  if (kv->n_layers < 1 || kv->n_pages < 1 || kv->n_kv_heads < 1 || kv->page_size < 1 ||
      kv->head_dim < 8 || kv->head_dim % 8 != 0)
    return fail(SPEC_E_SHAPE, "bad page dimensions (head_dim must be a multiple of 8)");
  if (((reinterpret_cast<uintptr_t>(kv->k) | reinterpret_cast<uintptr_t>(kv->v)) & 15u) != 0)
    return fail(SPEC_E_SHAPE, "k and v must be 16-byte aligned");
  if ((double)kv->n_kv_heads * kv->page_size * (kv->head_dim / 8) > INT32_MAX)
    return fail(SPEC_E_SHAPE, "a page is too large");
  // a layer in elements; each factor is below 2^31, so cut off before the product can overflow
  const double elems = (double)kv->n_pages * kv->n_kv_heads * kv->page_size * kv->head_dim;
  if (elems > 4.0e15) return fail(SPEC_E_SHAPE, "a layer's cache is too large");
  const int64_t layer = (int64_t)kv->n_pages * kv->n_kv_heads * kv->page_size * kv->head_dim;
  if (kv->layer_stride % 8 != 0 || (kv->n_layers > 1 && kv->layer_stride < layer))
    return fail(SPEC_E_SHAPE, "layer_stride must be a multiple of 8 and hold a layer's pages");
  if ((double)kv->layer_stride * kv->n_layers > 4.0e15) return fail(SPEC_E_SHAPE, "the cache is too large");
  if (book) {
    if (kv->table == nullptr || kv->len == nullptr) return fail(SPEC_E_INVALID, "null table or len");
    if (kv->n_slots < 1 || kv->max_pages < 1) return fail(SPEC_E_SHAPE, "n_slots and max_pages >= 1 required");
    if ((int64_t)kv->max_pages * kv->page_size > INT32_MAX)
      return fail(SPEC_E_SHAPE, "max_pages * page_size must stay below 2^31 positions");
  }
  return SPEC_OK;
}

static int check_refs(const spec_pages* kv) {
  if (kv->refs == nullptr)
    return fail(SPEC_E_UNSUPPORTED, "these pages are fixed to their slots (refs is NULL)");
  return SPEC_OK;
}

extern "C" int spec_pages_copy(const spec_pages* kv, int n, const int32_t* src, const int32_t* dst,
                               const int32_t* n_pos, int32_t* status, void* stream) {
  int rc = check_pages(kv, false);
  if (rc == SPEC_OK) rc = check_list(src, status, n);
  if (rc == SPEC_OK) rc = check_list(dst, status, n);
  if (rc != SPEC_OK) return rc;
  const int blocks = (int)((page_units(kv) + CP_UNITS - 1) / CP_UNITS);
  const double grid = 2.0 * n * kv->n_layers * blocks;
  if (grid > INT32_MAX) return fail(SPEC_E_SHAPE, "n * n_layers * page too large");
  pages_copy_kernel<<<(unsigned)grid, PG_THREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      *kv, n, src, dst, n_pos, blocks, status);
  return launched("page copy");
}

extern "C" int spec_pages_fork(const spec_pages* kv, int n, const int32_t* src, const int32_t* dst,
                               int32_t* status, void* stream) {
  int rc = check_pages(kv, true);
  if (rc == SPEC_OK) rc = check_refs(kv);
  if (rc == SPEC_OK) rc = check_list(src, status, n);
  if (rc == SPEC_OK) rc = check_list(dst, status, n);
  if (rc != SPEC_OK) return rc;
  pages_fork_kernel<<<n, PG_THREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(*kv, n, src, dst,
                                                                                 status);
  return launched("page fork");
}

extern "C" int spec_pages_extend(const spec_pages* kv, int n, const int32_t* slots,
                                 const int32_t* n_new, int32_t* copies, int32_t* status,
                                 void* stream) {
  int rc = check_pages(kv, true);
  if (rc == SPEC_OK) rc = check_refs(kv);
  if (rc == SPEC_OK) rc = check_list(slots, status, n);
  if (rc == SPEC_OK && (n_new == nullptr || copies == nullptr)) rc = fail(SPEC_E_INVALID, "null argument");
  if (rc != SPEC_OK) return rc;
  if (n > EX_THREADS) return fail(SPEC_E_SHAPE, "n must be <= 1024");
  const int64_t grid = (int64_t)n * kv->n_layers;
  if (grid > INT32_MAX) return fail(SPEC_E_SHAPE, "n * n_layers too large");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  pages_extend_kernel<<<1, EX_THREADS, 0, st>>>(*kv, n, slots, n_new, copies, status);
  rc = launched("page extend");
  if (rc != SPEC_OK) return rc;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = programmatic_launch() ? 1 : 0;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(PG_THREADS);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, pages_cow_kernel, *kv, slots, (const int32_t*)copies);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, std::string("page extend: ") + cudaGetErrorString(e));
  return SPEC_OK;
}

extern "C" int spec_pages_commit(const spec_pages* kv, int n, const int32_t* slots, int nt,
                                 const uint16_t* k_new, const uint16_t* v_new,
                                 int64_t new_layer_stride, const int32_t* path,
                                 const int32_t* n_path, int32_t* new_len, int32_t* status,
                                 void* stream) {
  int rc = check_pages(kv, true);
  if (rc == SPEC_OK) rc = check_list(slots, status, n);
  if (rc == SPEC_OK && (k_new == nullptr || v_new == nullptr || n_path == nullptr))
    rc = fail(SPEC_E_INVALID, "null argument");
  if (rc != SPEC_OK) return rc;
  if (nt < 1) return fail(SPEC_E_SHAPE, "nt >= 1 required");
  if (((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15u) != 0)
    return fail(SPEC_E_SHAPE, "k_new and v_new must be 16-byte aligned");
  const double rows = (double)n * nt * kv->n_kv_heads * kv->head_dim;
  if (rows > 4.0e15 || (double)new_layer_stride * kv->n_layers > 4.0e15)
    return fail(SPEC_E_SHAPE, "k_new / v_new are too large");
  const int64_t layer = (int64_t)n * nt * kv->n_kv_heads * kv->head_dim;
  if (new_layer_stride == 0) new_layer_stride = layer;
  if (new_layer_stride % 8 != 0 || (kv->n_layers > 1 && new_layer_stride < layer))
    return fail(SPEC_E_SHAPE, "new_layer_stride must be a multiple of 8 and hold a layer's rows");
  const int blocks = (nt + CM_ROWS - 1) / CM_ROWS;
  const double grid = (double)n * kv->n_layers * blocks;
  if (grid > INT32_MAX) return fail(SPEC_E_SHAPE, "n * n_layers * nt too large");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // lengths written where they are read from go up in a kernel behind
  const uintptr_t a = reinterpret_cast<uintptr_t>(kv->len), b = reinterpret_cast<uintptr_t>(new_len);
  const uintptr_t bytes = (uintptr_t)kv->n_slots * sizeof(int32_t);
  const bool in_place = new_len == nullptr || a == b;
  if (!in_place && a < b + bytes && b < a + bytes)
    return fail(SPEC_E_INVALID, "new_len overlaps len without being len");
  pages_commit_kernel<<<(unsigned)grid, PG_THREADS, 0, st>>>(*kv, n, slots, nt, k_new, v_new,
                                                             new_layer_stride, path, n_path,
                                                             in_place ? nullptr : new_len, blocks,
                                                             status);
  if (in_place)
    pages_advance_kernel<<<(n + 127) / 128, 128, 0, st>>>(n, slots, n_path,
                                                          kv->len, status);
  return launched("page commit");
}

extern "C" int spec_pages_free(const spec_pages* kv, int n, const int32_t* slots, int32_t* status,
                               void* stream) {
  int rc = check_pages(kv, true);
  if (rc == SPEC_OK) rc = check_refs(kv);
  if (rc == SPEC_OK) rc = check_list(slots, status, n);
  if (rc != SPEC_OK) return rc;
  pages_free_kernel<<<n, PG_THREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(*kv, n, slots,
                                                                                 status);
  return launched("page free");
}

extern "C" int spec_accept_tree(const int32_t* argmax, const int32_t* tokens, const int32_t* parents,
                                const int32_t* n_nodes, int n_seq, int nt, int32_t* path,
                                int32_t* n_path, int32_t* emitted, void* stream) {
  if (argmax == nullptr || tokens == nullptr || parents == nullptr || path == nullptr ||
      n_path == nullptr || emitted == nullptr)
    return fail(SPEC_E_INVALID, "null argument");
  if (n_seq < 1 || nt < 1 || nt > SPEC_MAX_TREE)
    return fail(SPEC_E_SHAPE, "n_seq >= 1 and nt in [1, 64] required");
  accept_tree_kernel<<<(n_seq + AT_WARPS - 1) / AT_WARPS, AT_WARPS * 32, 0,
                       reinterpret_cast<cudaStream_t>(stream)>>>(
      argmax, tokens, parents, n_nodes, n_seq, nt, path, n_path, emitted);
  return launched("tree accept");
}
