// cache.cu -- upkeep of a paged K/V cache on the device: forking and re-ordering
// sequences, reserving pages for coming tokens (with copy-on-write of a shared
// last page), the slots of those tokens, keeping the accepted nodes of a draft
// tree, closing the holes of the pool.  include/attn_fwd.h states the rules; all of them read and write
// lengths, tables and reference counts in device memory, so that a serving loop
// needs no round trip to the host.
//
// Two kinds of kernels:
//  * bookkeeping on some thousands of integers: latency bound, so each entry
//    point does it in one launch of few dependent steps.  Counts of pages are
//    kept in shared memory by the CTA that owns the page range (no global
//    atomics, the order of additions does not matter for integers), ranks of
//    free or live pages come from block-wide scans.
//  * moving K/V rows or pages: memory bound, 16 bytes per thread and access, with
//    several independent accesses in flight per thread.
#include "host.h"
#include "launch.h"
#include "pages.h"
#include "ptx.cuh"

#include <algorithm>
#include <cstdio>
#include <initializer_list>

using namespace attn;

namespace {

constexpr int kRange = 8192;     // pages counted at a time in shared memory
constexpr int kMaxSeqs = 8192;   // sequences per call
constexpr int kMaxCtas = 152;
constexpr int kChunk = 16384;    // bytes of a page that a CTA copies at a time

__device__ __forceinline__ void report(unsigned int* err) {
  if (err) atomicOr(err, 1u << kErrCacheBadIndex);
}

// refs_out[p] = refs[p] + the weights of the table entries that name page p, for
// this CTA's share of the pages.  span(b, begin, end) gives the entries
// [begin, end) of row b that count and their weight (0: none).  Every CTA reads
// all counted entries, a warp a run of 128 of one row.  cnt: kRange ints.
template <class Span>
__device__ void update_refs(const int32_t* refs, int32_t* refs_out, const int32_t* table, int B,
                            int max_pages, int num_pages, int cta, int ctas, int* cnt, unsigned int* err,
                            Span span) {
  const int per = (num_pages + ctas - 1) / ctas;
  const int p_end = min(num_pages, (cta + 1) * per);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int runs = (max_pages + 127) / 128;
  for (int p0 = cta * per; p0 < p_end; p0 += kRange) {
    const int n = min(kRange, p_end - p0);
    for (int i = threadIdx.x; i < n; i += blockDim.x) cnt[i] = refs[p0 + i];
    __syncthreads();
    for (int64_t task = warp; task < static_cast<int64_t>(B) * runs; task += warps) {
      const int b = static_cast<int>(task / runs), j0 = static_cast<int>(task - static_cast<int64_t>(b) * runs) * 128;
      int begin, end;
      const int weight = span(b, begin, end);
      if (weight == 0) continue;
      for (int j = max(begin, j0) + lane; j < min(end, j0 + 128); j += 32) {
        const int p = table[static_cast<int64_t>(b) * max_pages + j];
        if (p < 0 || p >= num_pages) {
          if (cta == 0) report(err);
        } else if (p >= p0 && p < p0 + n) {
          atomicAdd(&cnt[p - p0], weight);
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) refs_out[p0 + i] = cnt[i];
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Re-order: new sequence b is old sequence index[b].
struct ReorderParams {
  const int32_t *table, *seqlens, *refs, *index;
  int32_t *table_out, *seqlens_out, *refs_out;
  int B_in, B_out, max_pages, num_pages, page_log2;
  unsigned int* err;
};

__global__ void __launch_bounds__(512) reorder_kernel(const ReorderParams p) {
  extern __shared__ int sh[];
  pdl_launch_dependents();
  pdl_wait();
  int* cnt = sh;             // [kRange]
  int* times = sh + kRange;  // [B_in]: how often an old sequence is taken
  for (int b = threadIdx.x; b < p.B_in; b += blockDim.x) times[b] = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < p.B_out; b += blockDim.x) {
    const int i = p.index[b];
    if (i >= 0 && i < p.B_in) atomicAdd(&times[i], 1);
    else if (i != -1 && blockIdx.x == 0) report(p.err);
  }
  __syncthreads();
  // Rows of the new table, a warp a row.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int b = blockIdx.x * warps + warp; b < p.B_out; b += gridDim.x * warps) {
    int i = p.index[b];
    if (i < 0 || i >= p.B_in) i = -1;
    const int len = i >= 0 ? p.seqlens[i] : 0;
    const int held = held_pages(len, p.page_log2, p.max_pages);
    for (int j = lane; j < p.max_pages; j += 32)
      p.table_out[static_cast<int64_t>(b) * p.max_pages + j] =
          j < held ? p.table[static_cast<int64_t>(i) * p.max_pages + j] : -1;
    if (lane == 0) p.seqlens_out[b] = len;
  }
  update_refs(p.refs, p.refs_out, p.table, p.B_in, p.max_pages, p.num_pages, blockIdx.x, gridDim.x, cnt, p.err,
              [&](int b, int& begin, int& end) {
                const int w = times[b] - 1;
                begin = 0;
                end = w != 0 ? held_pages(p.seqlens[b], p.page_log2, p.max_pages) : 0;
                return w;
              });
}

// ---------------------------------------------------------------------------
// Block-wide exclusive sum of v; total in `all`.  scratch: 32 values.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* scratch, T& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  T pre = 0;
  all = 0;
  for (int i = 0; i < warps; ++i) {
    const T x = scratch[i];
    pre += i < warp ? x : 0;
    all += x;
  }
  return pre + inc - v;
}

// Eight consecutive reference counts, -1 past the end.
__device__ __forceinline__ void load8(const int32_t* refs, int p, int n, int (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p + i < n ? refs[p + i] : -1;
}

// ---------------------------------------------------------------------------
// Page copies.  A pool is [layers][num_pages][page bytes].
struct PoolParams {
  uint8_t *k, *v;
  int64_t page_bytes, layer_bytes;
  int layers;
};

// Bytes [off, off + n) of page src to page dst of one pool and layer; n a
// multiple of 16, by a group of kCopiers threads.  Eight 16-byte loads per thread
// go out before the first store.
constexpr int kCopiers = 128;
__device__ __forceinline__ void copy_chunk(const uint8_t* src, uint8_t* dst, int n) {
  constexpr int U = 8;
  const int tid = threadIdx.x & (kCopiers - 1);
  for (int i0 = 0; i0 < n; i0 += kCopiers * 16 * U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + (u * kCopiers + tid) * 16;
      if (i < n) x[u] = __ldcs(reinterpret_cast<const uint4*>(src + i));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + (u * kCopiers + tid) * 16;
      if (i < n) __stcs(reinterpret_cast<uint4*>(dst + i), x[u]);
    }
  }
}

// Task t of the copies of one page pair: layer, pool and chunk.
__device__ __forceinline__ void copy_task(const PoolParams& q, int src, int dst, int t, int chunks) {
  const int chunk = t % chunks, lk = t / chunks;
  uint8_t* pool = (lk & 1) ? q.v : q.k;
  const int64_t base = (lk >> 1) * q.layer_bytes + static_cast<int64_t>(chunk) * kChunk;
  const int n = static_cast<int>(q.page_bytes - static_cast<int64_t>(chunk) * kChunk < kChunk
                                     ? q.page_bytes - static_cast<int64_t>(chunk) * kChunk
                                     : kChunk);
  copy_chunk(pool + base + src * q.page_bytes, pool + base + dst * q.page_bytes, n);
}

// ---------------------------------------------------------------------------
// Reserve.
struct ReserveParams {
  const int32_t *table, *seqlens, *refs, *add;
  int32_t *table_out, *seqlens_out, *refs_out, *free_out;
  int B, max_pages, num_pages, page_log2;
  unsigned int* err;
};

// Sequences are taken in order.  One that grows out of a partly filled last
// page with other holders left copies it (the first `refs - 1` growers of a
// page do, the last holder keeps it).  New pages are the free pages in rising
// order, dealt to the sequences in order.  All or nothing.  Every CTA works the
// plan out for itself, which is short where sequences are some hundreds; a second
// kernel for the copies would have to wait for the first (64 beams, 16 layers:
// 47.9 us with two kernels, 45.1 with one; four beams 15.4 and 13.3).  The search
// for earlier holders of a page is quadratic in the sequences: the call takes 10
// us at 64, 12 at 256, 25 at 1024, 192 at 4096 and 670 at 8192 (pages of 64, no
// page shared; 4 to 10 us more where pairs share their pages and one of each
// copies).  CTA 0 writes the new pages and the counts, and all share the rows of
// the table (one CTA alone writes a 2 MB table in 50 us) and the copies: eight
// groups of 128 threads a CTA, 16 KB a task.
__global__ void __launch_bounds__(1024, 1) reserve_kernel(const ReserveParams p, const PoolParams q, int chunks) {
  extern __shared__ int sh[];
  int* last = sh;              // [B] page that the sequence would share, or -1
  int* start = sh + p.B;       // [B] first new page's number; then one past the end
  int* first = sh + 2 * p.B + 1;  // [B] first new column
  int* fresh = sh + 3 * p.B + 1;  // [B] first new page
  int* copiers = sh + 4 * p.B + 1;  // [B] the sequences that copy, in order
  __shared__ int scratch[32];
  __shared__ long long wide[32];
  const int tid = threadIdx.x, n_thr = blockDim.x;
  pdl_launch_dependents();
  pdl_wait();
  for (int b = tid; b < p.B; b += n_thr) {
    const int len = max(p.seqlens[b], 0), add = p.add[b];
    const int has = held_pages(len, p.page_log2, p.max_pages);
    int page = -1;
    if (add > 0 && (len & ((1 << p.page_log2) - 1)) != 0 && has == pages_of(len, p.page_log2)) {
      page = p.table[static_cast<int64_t>(b) * p.max_pages + has - 1];
      if (page < 0 || page >= p.num_pages) {
        report(p.err);
        page = -1;
      }
    }
    last[b] = page;
  }
  __syncthreads();
  long long total = 0;  // (thousands of long rows pass 32 bits; no pool holds them, but the answer says so)
  int copying = 0;   // sequences that copy
  bool bad = false;  // a sequence outgrows its row of the table: nothing is reserved
  for (int b0 = 0; b0 < p.B; b0 += n_thr) {
    const int b = b0 + tid;
    long long need = 0;
    int col = 0, copied = 0;
    if (b < p.B) {
      const int len = max(p.seqlens[b], 0), add = max(p.add[b], 0);
      const int has = held_pages(len, p.page_log2, p.max_pages);
      const int64_t want = (static_cast<int64_t>(len) + add + (1 << p.page_log2) - 1) >> p.page_log2;
      if (last[b] >= 0) {
        int before = 0;
        for (int i = 0; i < b; ++i) before += last[i] == last[b];
        copied = p.refs[last[b]] - before > 1;
      }
      if (p.add[b] < 0) report(p.err);
      col = has - copied;
      if (want > p.max_pages) bad = true;
      need = want > p.max_pages || want < col ? 0 : want - col;
    }
    long long all;
    const long long pre = block_scan(need, wide, all);
    if (b < p.B) {
      start[b] = static_cast<int>(total + pre);  // (read only where the total fits the pool)
      first[b] = col;
    }
    total += all;
    if (__syncthreads_or(copied)) {
      int n;
      const int k = copying + block_scan(copied, scratch, n);
      if (copied) copiers[k] = b;
      copying += n;
    }
  }
  if (tid == 0) start[p.B] = static_cast<int>(total);
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && blockIdx.x == 0) report(p.err);
  // Free pages there are.
  int free_pages = 0;
  for (int p0 = 0; p0 < p.num_pages; p0 += n_thr * 8) {
    int v[8], c = 0;
    load8(p.refs, p0 + tid * 8, p.num_pages, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) c += v[i] == 0;
    free_pages += c;
  }
  {
    int all;
    block_scan(free_pages, scratch, all);
    free_pages = all;
  }
  const bool fits = !bad && total <= free_pages;
  if (tid == 0 && blockIdx.x == 0) {
    const long long left = free_pages - total;
    *p.free_out = bad ? -p.num_pages - 1 : static_cast<int>(left > -0x7fffffffLL ? left : -0x7fffffffLL);
  }
  // Tables as they were, without the columns that get new pages.
  const int warp = tid >> 5, lane = tid & 31, warps = n_thr >> 5;
  for (int b = blockIdx.x * warps + warp; b < p.B; b += gridDim.x * warps) {
    const int len = max(p.seqlens[b], 0);
    const int has = held_pages(len, p.page_log2, p.max_pages);
    const int keep = fits ? min(has, first[b]) : has;
    const int want = fits ? start[b + 1] - start[b] + first[b] : has;
    for (int j = lane; j < p.max_pages; j += 32)
      if (j < keep || j >= want)
        p.table_out[static_cast<int64_t>(b) * p.max_pages + j] =
            j < keep ? p.table[static_cast<int64_t>(b) * p.max_pages + j] : -1;
    if (lane == 0) p.seqlens_out[b] = len + (fits ? max(p.add[b], 0) : 0);
  }
  const bool writer = blockIdx.x == 0;
  if (!writer && !(fits && copying > 0)) return;
  // Deal the free pages out and write the counts.
  int rank0 = 0;
  for (int p0 = 0; p0 < p.num_pages; p0 += n_thr * 8) {
    int v[8], c = 0;
    const int q0 = p0 + tid * 8;
    load8(p.refs, q0, p.num_pages, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) c += v[i] == 0;
    int all;
    int k = rank0 + block_scan(c, scratch, all);
    rank0 += all;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (q0 + i >= p.num_pages) break;
      int refs = v[i];
      if (v[i] == 0) {
        if (fits && k < total) {
          int lo = 0, hi = p.B - 1;  // the sequence with start <= k < its end
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] <= k) lo = mid;
            else hi = mid - 1;
          }
          if (k == start[lo]) fresh[lo] = q0 + i;
          if (writer)
            p.table_out[static_cast<int64_t>(lo) * p.max_pages + first[lo] + (k - start[lo])] = q0 + i;
          refs = 1;
        }
        ++k;
      }
      if (writer) p.refs_out[q0 + i] = refs;
    }
  }
  __syncthreads();
  if (!fits) return;
  if (writer)  // the copied pages have one holder less
    for (int i = tid; i < copying; i += n_thr) atomicSub(&p.refs_out[last[copiers[i]]], 1);
  const int per = chunks * 2 * q.layers, groups = n_thr / kCopiers;
  const int64_t tasks = static_cast<int64_t>(copying) * per;
  for (int64_t task = static_cast<int64_t>(tid / kCopiers) * gridDim.x + blockIdx.x; task < tasks;
       task += static_cast<int64_t>(groups) * gridDim.x) {
    const int64_t i = task / per;
    const int b = copiers[i];
    copy_task(q, last[b], fresh[b], static_cast<int>(task - i * per), chunks);
  }
}

// ---------------------------------------------------------------------------
// Accept: the rows of the accepted nodes move to the front of the tree's rows.
struct AcceptParams {
  const int32_t *table, *seqlens, *refs, *path, *path_lens, *tree_lens;
  int32_t *seqlens_out, *refs_out;
  int B, A, T, max_pages, num_pages, page_log2, ref_ctas, row_ctas;
  int64_t row_bytes;
  unsigned int* err;
};

// Nodes of sequence b in the cache, and its base position.
__device__ __forceinline__ int accept_tree(const AcceptParams& p, int b, int& base) {
  const int L = max(0, min(p.seqlens[b], p.max_pages << p.page_log2));
  int n = p.tree_lens != nullptr ? max(0, min(p.tree_lens[b], p.T)) : p.T;
  n = min(n, L);
  base = L - n;
  return n;
}

// Accepted nodes: the longest prefix of the path that rises strictly within the
// tree (anything else is an error).  A warp computes it.
__device__ __forceinline__ int accept_count(const AcceptParams& p, int b, int n) {
  const int lane = threadIdx.x & 31;
  const int want = p.path_lens[b], m = max(0, min(want, p.A));
  int good = m;
  for (int i0 = 0; i0 < m; i0 += 32) {
    const int i = i0 + lane;
    bool ok = true;
    if (i < m) {
      const int x = p.path[static_cast<int64_t>(b) * p.A + i];
      const int before = i > 0 ? p.path[static_cast<int64_t>(b) * p.A + i - 1] : -1;
      ok = x > before && x >= 0 && x < n;
    }
    const unsigned no = __ballot_sync(0xffffffffu, !ok);
    if (no != 0) {
      good = i0 + __ffs(no) - 1;
      break;
    }
  }
  if (good != want && lane == 0) report(p.err);
  return good;
}

// Blocks [0, ref_ctas): counts and lengths.  The others: one (sequence, layer, pool,
// part of the row) each.  A thread owns 16 bytes of the row and moves them for
// every accepted node in order: node path[i] >= i goes to row i, and because the
// path rises no later source is overwritten, so loads of several nodes may go
// out ahead of the stores.
__global__ void __launch_bounds__(128) accept_kernel(const AcceptParams p, const PoolParams q) {
  extern __shared__ int sh[];
  pdl_launch_dependents();
  pdl_wait();
  if (static_cast<int>(blockIdx.x) < p.ref_ctas) {
    int* cnt = sh;
    int* keep = sh + kRange;  // [B] new length
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {  // (a warp each would take B / 4 round trips)
      int base;
      const int n = accept_tree(p, b, base);
      const int m = max(0, min(p.path_lens[b], p.A));
      int good = m, before = -1;
#pragma unroll 8
      for (int i = 0; i < m; ++i) {
        const int x = p.path[static_cast<int64_t>(b) * p.A + i];
        if (!(x > before && x < n)) good = min(good, i);
        before = x;
      }
      keep[b] = base + good;
      if (blockIdx.x == 0) p.seqlens_out[b] = base + good;
    }
    __syncthreads();
    update_refs(p.refs, p.refs_out, p.table, p.B, p.max_pages, p.num_pages, blockIdx.x, p.ref_ctas, cnt, p.err,
                [&](int b, int& begin, int& end) {
                  begin = pages_of(keep[b], p.page_log2);
                  end = held_pages(p.seqlens[b], p.page_log2, p.max_pages);
                  return begin < end ? -1 : 0;
                });
    return;
  }
  int task = blockIdx.x - p.ref_ctas;
  const int part = task % p.row_ctas;
  task /= p.row_ctas;
  const int lk = task % (2 * q.layers), b = task / (2 * q.layers);
  int base;
  const int n = accept_tree(p, b, base);
  const int m = accept_count(p, b, n);
  const int64_t col = (static_cast<int64_t>(part) * blockDim.x + threadIdx.x) * 16;
  if (col >= p.row_bytes) return;
  uint8_t* pool = ((lk & 1) ? q.v : q.k) + (lk >> 1) * q.layer_bytes + col;
  const int32_t* row = p.table + static_cast<int64_t>(b) * p.max_pages;
  auto at = [&](int pos) -> uint8_t* {  // nullptr behind a bad table entry
    const int page = row[pos >> p.page_log2];
    if (page < 0 || page >= p.num_pages) {
      report(p.err);
      return nullptr;
    }
    return pool + page * q.page_bytes + (pos & ((1 << p.page_log2) - 1)) * p.row_bytes;
  };
  constexpr int U = 8;
  for (int i0 = 0; i0 < m; i0 += U) {
    uint4 x[U];
    uint8_t* dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      dst[u] = nullptr;
      if (i0 + u < m) {
        const int node = p.path[static_cast<int64_t>(b) * p.A + i0 + u];
        if (node != i0 + u) {  // (a node already in place stays)
          const uint8_t* src = at(base + node);
          if (src != nullptr) {
            x[u] = *reinterpret_cast<const uint4*>(src);
            dst[u] = at(base + i0 + u);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] != nullptr) *reinterpret_cast<uint4*>(dst[u]) = x[u];
  }
}

// ---------------------------------------------------------------------------
// Compact: live pages past the count of live pages move into the holes before it.
struct CompactParams {
  const int32_t *table, *seqlens, *refs;
  int32_t *table_out, *refs_out, *map;
  int32_t *moved;  // [0]: pages that move, then their numbers
  int B, max_pages, num_pages, page_log2;
  unsigned int* err;
};

constexpr int kOnePass = 8192;  // eight pages for each of 1024 threads

__global__ void __launch_bounds__(1024) compact_plan_kernel(const CompactParams p) {
  __shared__ int scratch[32];
  const int tid = threadIdx.x, n_thr = blockDim.x;
  pdl_launch_dependents();
  pdl_wait();
  if (p.num_pages <= kOnePass) {
    // The counts fit the block's registers: one load and one scan.  With r(q)
    // the live pages before page q, hole q below `live` is number q - r(q), and
    // live page q above it moves as number r(q) - r(live).  There are as many
    // holes as moves, so at most kOnePass / 2.  (Against the passes below, whose
    // numbers go through global memory: a pool of 300 pages 10.3 -> 8.2 us, 4096
    // pages 96.1 -> 94.4, both with the moves.)
    __shared__ int hole[kOnePass / 2];
    __shared__ int before_live;
    const int q0 = tid * 8;
    int v[8], c = 0;
    load8(p.refs, q0, p.num_pages, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) c += v[i] > 0;
    int live;
    const int rank = block_scan(c, scratch, live);
    int r = rank;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (q0 + i == live) before_live = r;
      if (q0 + i < live && v[i] <= 0) hole[q0 + i - r] = q0 + i;
      r += v[i] > 0;
    }
    if (tid == 0 && live == kOnePass) before_live = live;  // (no thread has a page `live`)
    __syncthreads();
    const int base = before_live;
    r = rank;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = q0 + i;
      if (q >= p.num_pages) break;
      int to = v[i] > 0 ? q : -1;
      if (q >= live) {
        p.refs_out[q] = 0;
        if (v[i] > 0) {
          to = hole[r - base];
          p.moved[1 + r - base] = q;
        }
      }
      if (to >= 0) p.refs_out[to] = v[i];
      p.map[q] = to;
      r += v[i] > 0;
    }
    if (tid == 0) p.moved[0] = live - base;
    return;
  }
  int live = 0;
  for (int p0 = 0; p0 < p.num_pages; p0 += n_thr * 8) {
    int v[8];
    load8(p.refs, p0 + tid * 8, p.num_pages, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) live += v[i] > 0;
  }
  {
    int all;
    block_scan(live, scratch, all);
    live = all;
  }
  // Holes below `live`: the k-th is noted in refs_out[live + k] (there are as
  // many live pages above, and refs_out is written there last).
  int rank0 = 0;
  for (int p0 = 0; p0 < live; p0 += n_thr * 8) {
    int v[8], c = 0;
    const int q0 = p0 + tid * 8;
    load8(p.refs, q0, live, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) c += q0 + i < live && v[i] <= 0;
    int all;
    int k = rank0 + block_scan(c, scratch, all);
    rank0 += all;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (q0 + i >= live) break;
      if (v[i] > 0) {
        p.refs_out[q0 + i] = v[i];
        p.map[q0 + i] = q0 + i;
      } else {
        p.refs_out[live + k++] = q0 + i;
        p.map[q0 + i] = -1;
      }
    }
  }
  __syncthreads();
  rank0 = 0;
  for (int p0 = live; p0 < p.num_pages; p0 += n_thr * 8) {
    int v[8], c = 0;
    const int q0 = p0 + tid * 8;
    load8(p.refs, q0, p.num_pages, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) c += v[i] > 0;
    int all;
    int k = rank0 + block_scan(c, scratch, all);
    rank0 += all;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (q0 + i >= p.num_pages) break;
      int to = -1;
      if (v[i] > 0) {
        p.moved[1 + k] = q0 + i;
        to = p.refs_out[live + k++];
        p.refs_out[to] = v[i];
      }
      p.map[q0 + i] = to;
    }
  }
  if (tid == 0) p.moved[0] = rank0;
  __syncthreads();
  for (int i = live + tid; i < p.num_pages; i += n_thr) p.refs_out[i] = 0;
}

__global__ void __launch_bounds__(128) compact_move_kernel(const CompactParams p, const PoolParams q, int chunks) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t entries = static_cast<int64_t>(p.B) * p.max_pages;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < entries;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int b = static_cast<int>(i / p.max_pages), j = static_cast<int>(i - static_cast<int64_t>(b) * p.max_pages);
    int to = -1;
    if (j < held_pages(p.seqlens[b], p.page_log2, p.max_pages)) {
      const int page = p.table[i];
      if (page >= 0 && page < p.num_pages) to = p.map[page];
      if (to < 0) report(p.err);
    }
    p.table_out[i] = to;
  }
  const int per = chunks * 2 * q.layers;
  const int64_t tasks = static_cast<int64_t>(p.moved[0]) * per;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int64_t k = task / per;
    const int page = p.moved[1 + k];
    copy_task(q, page, p.map[page], static_cast<int>(task - k * per), chunks);
  }
}

// ---------------------------------------------------------------------------
// Slot map: where the new tokens of every sequence go, in packed order.  Latency
// bound: one launch, each CTA sums the counts for itself (8192 of them: 16 rounds
// of the block) and finds its tokens' sequences by bisection in shared memory.  64 tokens
// 2.6 us, 66,000 of 256 sequences 3.6.
struct SlotsParams {
  const int32_t *table, *seqlens, *add;
  int32_t *slots, *positions, *cu, *sequence;
  int B, N, max_pages, num_pages, page_log2;
  unsigned int* err;
};

constexpr int kSlotTokens = 1024;  // tokens per CTA

__global__ void __launch_bounds__(512) slots_kernel(const SlotsParams p) {
  extern __shared__ int cu[];  // [B + 1], none above N
  __shared__ long long scratch[32];
  pdl_launch_dependents();
  pdl_wait();
  bool bad = false;
  long long before = 0;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const int n = b < p.B ? p.add[b] : 0;
    bad |= n < 0;
    long long all;
    const long long at = before + block_scan<long long>(max(n, 0), scratch, all);
    if (b < p.B) cu[b] = static_cast<int>(min(at, static_cast<long long>(p.N)));
    before += all;
  }
  if (threadIdx.x == 0) cu[p.B] = static_cast<int>(min(before, static_cast<long long>(p.N)));
  __syncthreads();
  if (blockIdx.x == 0) {
    if (bad || (threadIdx.x == 0 && before > p.N)) report(p.err);
    for (int b = threadIdx.x; b <= p.B; b += blockDim.x) p.cu[b] = cu[b];
  }
  const int total = cu[p.B];
  const int t0 = blockIdx.x * kSlotTokens, t1 = min(p.N, t0 + kSlotTokens);
  for (int t = t0 + threadIdx.x; t < t1; t += blockDim.x) {
    int slot = -1, position = 0, b = -1;
    if (t < total) {
      int lo = 0, hi = p.B;  // cu[lo] <= t < cu[hi]
      while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (cu[m] <= t) lo = m;
        else hi = m;
      }
      b = lo;
      const long long pos = static_cast<long long>(p.seqlens[b]) - p.add[b] + (t - cu[b]);
      if (pos >= 0 && (pos >> p.page_log2) < p.max_pages) {
        position = static_cast<int>(pos);
        const int page = p.table[static_cast<int64_t>(b) * p.max_pages + (position >> p.page_log2)];
        if (page >= 0 && page < p.num_pages)
          slot = (page << p.page_log2) + (position & ((1 << p.page_log2) - 1));
      }
      if (slot < 0) report(p.err);
    }
    p.slots[t] = slot;
    p.positions[t] = position;
    p.sequence[t] = b;
  }
}

// ---------------------------------------------------------------------------
bool page_size_ok(int s) { return s == 16 || s == 32 || s == 64 || s == 128 || s == 256; }
int log2_of(int s) {
  int l = 0;
  while ((1 << l) < s) ++l;
  return l;
}

// Sizes, and the tables that must be there: `ints` always, `rows` where there are
// sequences.
attn_status check_cache(int B, int max_pages, int num_pages, int page_size, std::initializer_list<const void*> ints,
                        std::initializer_list<const void*> rows) {
  if (B < 0 || max_pages <= 0 || num_pages <= 0) return ATTN_ERR_INVALID;
  if (!page_size_ok(page_size) || B > kMaxSeqs) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_pages) * page_size > 0x7fffffffLL ||
      static_cast<int64_t>(max_pages) * page_size > 0x7fffffffLL)
    return ATTN_ERR_UNSUPPORTED;
  for (const void* p : ints)
    if (p == nullptr || !host_aligned(p, 4)) return ATTN_ERR_INVALID;
  if (B > 0)
    for (const void* p : rows)
      if (p == nullptr || !host_aligned(p, 4)) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

attn_status check_pool(const void* k, const void* v, int layers, int64_t row_bytes) {
  if (layers <= 0 || row_bytes <= 0 || row_bytes % 16 != 0 || row_bytes > (1 << 24)) return ATTN_ERR_INVALID;
  if (k == nullptr || v == nullptr || !host_aligned(k, 16) || !host_aligned(v, 16)) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

PoolParams pool_params(void* k, void* v, int layers, int64_t row_bytes, int page_size, int num_pages) {
  PoolParams q;
  q.k = static_cast<uint8_t*>(k);
  q.v = static_cast<uint8_t*>(v);
  q.page_bytes = row_bytes * page_size;
  q.layer_bytes = q.page_bytes * num_pages;
  q.layers = layers;
  return q;
}

int chunks_of(const PoolParams& q) { return static_cast<int>((q.page_bytes + kChunk - 1) / kChunk); }

// CTAs that count references: one per 1024 pages.
int ref_ctas(int num_pages) { return std::min(kMaxCtas, (num_pages + 1023) / 1024); }
// The same where they also write a table: at least one per 32768 entries.
int table_ctas(int B, int max_pages, int least) {
  const int64_t n = (static_cast<int64_t>(B) * max_pages + 32767) / 32768;
  return static_cast<int>(std::max<int64_t>(least, std::min<int64_t>(n, kMaxCtas)));
}

// Dynamic shared memory of a call over B sequences.
constexpr size_t reorder_smem(int B) { return (kRange + static_cast<size_t>(B)) * 4; }  // accept's too
constexpr size_t reserve_smem(int B) { return (5 * static_cast<size_t>(B) + 1) * 4; }
constexpr size_t slots_smem(int B) { return (static_cast<size_t>(B) + 1) * 4; }

}  // namespace

extern "C" {

attn_status attn_cache_reorder(const int32_t* block_table, const int32_t* seqlens, const int32_t* page_refs,
                               const int32_t* index, int32_t* table_out, int32_t* seqlens_out,
                               int32_t* refs_out, int B_in, int B_out, int max_pages, int num_pages,
                               int page_size, void* stream) {
  if (B_in < 0 || B_out < 0) return ATTN_ERR_INVALID;
  attn_status st = check_cache(B_in, max_pages, num_pages, page_size, {page_refs, refs_out}, {block_table, seqlens});
  if (st == ATTN_OK) st = check_cache(B_out, max_pages, num_pages, page_size, {}, {index, table_out, seqlens_out});
  if (st != ATTN_OK) return st;
  if (B_in > 0 && B_out > 0 && (table_out == block_table || seqlens_out == seqlens)) return ATTN_ERR_INVALID;
  ReorderParams p{block_table, seqlens, page_refs, index, table_out, seqlens_out, refs_out,
                  B_in, B_out, max_pages, num_pages, log2_of(page_size), nullptr};
  if (host_device_state(&p.err, nullptr) != ATTN_OK) return ATTN_ERR_CUDA;
  return host_finish(launch_pdl_upto<reorder_kernel>(reorder_smem(kMaxSeqs),
                                                     dim3(table_ctas(B_out, max_pages, ref_ctas(num_pages))), 512,
                                                     reorder_smem(B_in), static_cast<cudaStream_t>(stream), p),
                     "attn_cache_reorder");
}

attn_status attn_cache_reserve(void* k_pool, void* v_pool, const int32_t* block_table, const int32_t* seqlens,
                               const int32_t* page_refs, const int32_t* add, int32_t* table_out,
                               int32_t* seqlens_out, int32_t* refs_out, int32_t* free_out, int B,
                               int max_pages, int num_pages, int page_size, int layers, int64_t row_bytes,
                               void* stream) {
  attn_status st = check_cache(B, max_pages, num_pages, page_size,
                               {page_refs, refs_out, free_out},
                               {block_table, seqlens, add, table_out, seqlens_out});
  if (st != ATTN_OK) return st;
  st = check_pool(k_pool, v_pool, layers, row_bytes);
  if (st != ATTN_OK) return st;
  if ((B > 0 && (table_out == block_table || seqlens_out == seqlens)) || refs_out == page_refs)
    return ATTN_ERR_INVALID;
  ReserveParams p{block_table, seqlens, page_refs, add, table_out, seqlens_out, refs_out, free_out,
                  B, max_pages, num_pages, log2_of(page_size), nullptr};
  int sms = 0;
  if (host_device_state(&p.err, &sms) != ATTN_OK) return ATTN_ERR_CUDA;
  const PoolParams q = pool_params(k_pool, v_pool, layers, row_bytes, page_size, num_pages);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int chunks = chunks_of(q);
  const int64_t tasks = static_cast<int64_t>(B) * chunks * 2 * layers;
  const int grid = static_cast<int>(std::max<int64_t>(table_ctas(B, max_pages, 1), std::min<int64_t>(tasks, sms)));
  return host_finish(launch_pdl_upto<reserve_kernel>(reserve_smem(kMaxSeqs), dim3(grid), 1024, reserve_smem(B), s, p,
                                                     q, chunks),
                     "attn_cache_reserve");
}

attn_status attn_cache_accept(void* k_pool, void* v_pool, const int32_t* block_table, const int32_t* seqlens,
                              const int32_t* page_refs, const int32_t* path, const int32_t* path_lens,
                              const int32_t* tree_lens, int32_t* seqlens_out, int32_t* refs_out, int B, int A,
                              int T, int max_pages, int num_pages, int page_size, int layers,
                              int64_t row_bytes, void* stream) {
  if (A < 0 || T < 0) return ATTN_ERR_INVALID;
  attn_status st = check_cache(B, max_pages, num_pages, page_size,
                               {page_refs, refs_out}, {block_table, seqlens, path_lens, seqlens_out});
  if (st != ATTN_OK) return st;
  st = check_pool(k_pool, v_pool, layers, row_bytes);
  if (st != ATTN_OK) return st;
  if ((A > 0 && B > 0 && (path == nullptr || !host_aligned(path, 4))) || !host_aligned(tree_lens, 4) ||
      (B > 0 && seqlens_out == seqlens))
    return ATTN_ERR_INVALID;
  AcceptParams p{block_table, seqlens, page_refs, path, path_lens, tree_lens, seqlens_out, refs_out, B, A, T,
                 max_pages, num_pages, log2_of(page_size), ref_ctas(num_pages),
                 static_cast<int>((row_bytes + 2047) / 2048), row_bytes, nullptr};
  if (host_device_state(&p.err, nullptr) != ATTN_OK) return ATTN_ERR_CUDA;
  const PoolParams q = pool_params(k_pool, v_pool, layers, row_bytes, page_size, num_pages);
  const int64_t blocks = p.ref_ctas + static_cast<int64_t>(B) * 2 * layers * p.row_ctas;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  return host_finish(launch_pdl_upto<accept_kernel>(reorder_smem(kMaxSeqs), dim3(static_cast<unsigned>(blocks)), 128,
                                                    reorder_smem(B), static_cast<cudaStream_t>(stream), p, q),
                     "attn_cache_accept");
}

attn_status attn_cache_compact(void* k_pool, void* v_pool, const int32_t* block_table, const int32_t* seqlens,
                               const int32_t* page_refs, int32_t* table_out, int32_t* refs_out,
                               int32_t* page_map, int32_t* workspace, int B, int max_pages, int num_pages,
                               int page_size, int layers, int64_t row_bytes, void* stream) {
  attn_status st = check_cache(B, max_pages, num_pages, page_size,
                               {page_refs, refs_out, page_map, workspace}, {block_table, seqlens, table_out});
  if (st != ATTN_OK) return st;
  st = check_pool(k_pool, v_pool, layers, row_bytes);
  if (st != ATTN_OK) return st;
  if ((B > 0 && table_out == block_table) || refs_out == page_refs) return ATTN_ERR_INVALID;
  CompactParams p{block_table, seqlens, page_refs, table_out, refs_out, page_map, workspace,
                  B, max_pages, num_pages, log2_of(page_size), nullptr};
  int sms = 0;
  if (host_device_state(&p.err, &sms) != ATTN_OK) return ATTN_ERR_CUDA;
  const PoolParams q = pool_params(k_pool, v_pool, layers, row_bytes, page_size, num_pages);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), 1024, 0, s, p);
  if (e == cudaSuccess)
    e = launch_pdl(compact_move_kernel, dim3(8 * sms), 128, 0, s, p, q, chunks_of(q));
  return host_finish(e, "attn_cache_compact_plan+attn_cache_compact_move");
}

attn_status attn_cache_slots(const int32_t* block_table, const int32_t* seqlens, const int32_t* add, int32_t* slots,
                             int32_t* positions, int32_t* cu_seqlens, int32_t* sequence, int B, int num_tokens,
                             int max_pages, int num_pages, int page_size, void* stream) {
  if (num_tokens < 0) return ATTN_ERR_INVALID;
  attn_status st = check_cache(B, max_pages, num_pages, page_size, {cu_seqlens}, {block_table, seqlens, add});
  if (st != ATTN_OK) return st;
  for (const void* p : {slots, positions, sequence})
    if (num_tokens > 0 && (p == nullptr || !host_aligned(p, 4))) return ATTN_ERR_INVALID;
  SlotsParams p{block_table, seqlens, add, slots, positions, cu_seqlens, sequence, B, num_tokens,
                max_pages, num_pages, log2_of(page_size), nullptr};
  if (host_device_state(&p.err, nullptr) != ATTN_OK) return ATTN_ERR_CUDA;
  if (num_tokens > 0x7fffffff - kSlotTokens) return ATTN_ERR_UNSUPPORTED;
  const int grid = std::max(1, (num_tokens + kSlotTokens - 1) / kSlotTokens);
  return host_finish(launch_pdl_upto<slots_kernel>(slots_smem(kMaxSeqs), dim3(grid), 512, slots_smem(B),
                                                   static_cast<cudaStream_t>(stream), p),
                     "attn_cache_slots");
}

}  // extern "C"
