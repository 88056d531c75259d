// tree_kernel.cuh -- attention of a tree of drafted tokens over a paged K/V cache on
// sm_103a, compiled once per head dimension (tree_d64.cu, tree_d128.cu define
// ATTN_TREE_D and include this).
//
// Sequence b has L keys in the cache, the last n of them its drafted nodes
// (base = L - n).  Query i (node i) sees every key below base (with a window:
// keys >= base + depth_i - left, and the first sink_tokens) and the nodes whose
// bit is set in its mask row.  O, LSE as everywhere in this library.
//
// The work is one long read of K and V (4 Hq/Hkv T flops per byte pair of them:
// memory bound up to about 256 query rows per kv head), whatever the lengths:
//
//  * rows: the g = Hq / Hkv heads of a kv head share its tiles, qpt = 128 / g
//    whole queries per 128-row tile, row = query * g + head (the box of one
//    5-D tensor map; any g up to 128).
//  * one persistent CTA per SM.  The 128-key tiles of all (sequence, query
//    block, kv head) units form one line, and CTA c takes the tiles
//    [c T / G, (c + 1) T / G) of it, wherever sequence ends fall: every SM
//    reads the same number of bytes for any mix of lengths.  The lengths
//    live on the device, so each CTA finds its place by a scan.  A unit that
//    ends up on one CTA is finished there; of a unit cut in pieces each CTA
//    writes (m, l, unnormalised O) to the workspace (at most two pieces per
//    CTA: its first and its last) and a second kernel merges them.
//  * up to 128 rows per unit, one query tile is not enough to hide the chain
//    S -> softmax -> P.V behind the loads: the two softmax warpgroups then take
//    alternate K/V tiles of the unit, each with its own running maximum, sum
//    and O accumulator, merged from tensor memory at the unit's end.  Above
//    128 rows they take one query tile each and share every K/V tile.
//  * K and V tiles pass through one ring of shared-memory slots in consumption
//    order K0, K1, V0, K2, V1, ...; what Q does not take of shared memory is
//    ring (d = 128: 6 slots of 32 KB, or 5 beside two query tiles).
//  * only the tiles that hold drafted nodes, the sequence's end or a window's
//    edge are masked, from a 128-bit visibility word per row.
#pragma once
#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "softmax.cuh"

#include <type_traits>

namespace attn {

template <int D_>
struct TreeCfg {
  static constexpr int D = D_;
  static constexpr int BN = 128;                  // keys per tile
  static constexpr int NCHUNK = D / 64;           // 64-column swizzle atoms along d
  static constexpr int CHUNK_BYTES = BN * 128;
  static constexpr int TILE_BYTES = BN * D * 2;
  static constexpr int NBUF = D == 128 ? 7 : 13;  // tile buffers: 1 or 2 of Q, the rest ring
  // 8 softmax warps, the producer, the MMA issuer and two idle warps: setmaxnreg
  // works on whole warpgroups.  The launch's 384 x 168 registers are split
  // 256 x 192 + 128 x 120 (both 64512), as in the prefill kernel; launch_tree_t
  // checks the launch count, on which setmaxnreg.inc relies.
  static constexpr int THREADS = 384;
  static constexpr int LAUNCH_REGS = 168, SOFT_REGS = 192, OTHER_REGS = 120;
  static_assert(256 * SOFT_REGS + 128 * OTHER_REGS <= THREADS * LAUNCH_REGS, "register split");
  static constexpr uint32_t TM_COLS = 512;
  __device__ static constexpr uint32_t tm_s(int t) { return 128u * t; }
  __device__ static constexpr uint32_t tm_o(int t) { return 256u + D * t; }
};

template <class C>
struct TreeSmem {
  alignas(1024) uint8_t buf[C::NBUF][C::TILE_BYTES];
  uint64_t full[C::NBUF], empty[C::NBUF];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_half[2], p_full[2], o_final[2], o_free, xch, xread;
  uint64_t teardown;
  float2 x[2][128];     // (m, l) of a row, per warpgroup
  long long scan[16];
  uint32_t tmem_base;
  int abort_flag;
};

// What the kernel needs to know of one sequence.
struct TreeSeq {
  int L, base, n;     // keys, keys before the drafted nodes, nodes
  int nkeep, gap;     // tile of step k: k < nkeep ? k : k + gap
  int tiles;          // K/V tiles with a visible key
  int slots;          // its share of the work line per unit: max(tiles, 1)
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  s.L = max(0, min(p.seqlens_k[b], p.max_pages * p.page_size));
  s.n = p.tree_lens != nullptr ? max(0, min(p.tree_lens[b], p.T)) : p.T;
  s.n = min(s.n, s.L);
  s.base = s.L - s.n;
  const int jb = p.win_left >= 0 ? max(0, s.base - p.win_left) / 128 : 0;
  s.nkeep = min((min(p.sink_tokens, s.base) + 127) / 128, jb);
  s.gap = jb - s.nkeep;
  s.tiles = s.n > 0 ? (s.L + 127) / 128 - s.gap : 0;  // without a node nothing is asked
  s.slots = max(s.tiles, 1);
  return s;
}

// Block-wide scan over the sequences: the total number of tile slots of one
// unit per sequence, and the sequence whose slots hold unit-slot x of the line
// (x in [0, total * units)): cum is the slots before it.  Every thread returns
// the same values.  At most 14 warps; scratch: 16 long longs.
__device__ inline long long tree_total(const TreeParams& p, long long* scratch) {
  long long v = 0;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) v += tree_seq(p, b).slots;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  long long t = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) t += scratch[i];
  return t;
}

__device__ inline void tree_locate(const TreeParams& p, long long x, long long* scratch, int& b_out,
                                   long long& cum_out) {
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long before = 0;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const long long n = b < p.B ? tree_seq(p, b).slots : 0;
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    long long pre = before, all = before;
    for (int i = 0; i < warps; ++i) {
      if (i < warp) pre += scratch[i];
      all += scratch[i];
    }
    __syncthreads();
    const bool mine = b < p.B && (pre + inc - n) * p.units <= x && x < (pre + inc) * p.units;
    if (mine) {
      scratch[14] = b;
      scratch[15] = pre + inc - n;
    }
    __syncthreads();
    if (x < all * p.units) break;  // found in this chunk
    before = all;
  }
  b_out = static_cast<int>(scratch[14]);
  cum_out = scratch[15];
}

// CTAs that share a line of `line` tile slots, and the first slot of CTA c.
__device__ __forceinline__ int tree_ctas(const TreeParams& p, long long line) {
  const long long want = (line + p.min_share - 1) / p.min_share;
  return static_cast<int>(want < p.grid ? want : p.grid);
}

// A CTA's walk along the line, one segment (a run of tiles of one unit) at a time.
struct TreeWalk {
  int b, u, k;    // next sequence, unit within it, tile slot
  int rem;        // tile slots left
};
struct TreeSeg {
  TreeSeq q;
  int b, hk, m0;    // sequence, kv head, first query
  int k0, n;        // tile steps [k0, k0 + n) of the unit
  bool whole;       // the unit's only segment
  bool first;       // the CTA's first segment
};

__device__ __forceinline__ bool tree_next(const TreeParams& p, TreeWalk& w, TreeSeg& s, bool first) {
  if (w.rem <= 0) return false;
  s.q = tree_seq(p, w.b);
  const int take = min(w.rem, s.q.slots - w.k);
  s.b = w.b;
  const int rb = w.u / p.Hkv;
  s.hk = w.u - rb * p.Hkv;
  s.m0 = rb * (p.two_tiles ? 2 : 1) * p.qpt;
  s.k0 = w.k;
  s.n = s.q.tiles > 0 ? take : 0;
  s.whole = take == s.q.slots;
  s.first = first;
  w.rem -= take;
  w.k += take;
  if (w.k == s.q.slots) {
    w.k = 0;
    if (++w.u == p.units) {
      w.u = 0;
      ++w.b;
    }
  }
  return true;
}

__device__ __forceinline__ int tree_tile(const TreeSeq& q, int k) { return k < q.nkeep ? k : k + q.gap; }

// Item of K_i / V_i of an n-tile segment in the ring order K0, K1, V0, K2, V1, ...
__device__ __forceinline__ int tree_k_item(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int tree_v_item(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

// One K or V tile, page piece by page piece (box of min(page, 128) rows).  Pieces
// behind the sequence's end, without a visible key, or behind a bad table
// entry (an error) read one row past the pool: zeros.
template <class C>
__device__ __forceinline__ void tree_load_tile(const TreeParams& p, const TreeSeg& s, int tile,
                                               const CUtensorMap* map, uint8_t* dst, uint64_t* bar) {
  const int P = p.page_size, BR = min(P, C::BN);
  const int32_t* bt = p.block_table + static_cast<int64_t>(s.b) * p.max_pages;
  const int klo = p.win_left >= 0 ? max(0, s.q.base - p.win_left) : 0;
  for (int r0 = 0; r0 < C::BN; r0 += BR) {
    const int key = tile * C::BN + r0;
    int row = p.num_pages * P;
    if (key < s.q.L && (key + BR > klo || key < p.sink_tokens)) {
      const int lp = key / P;
      const int phys = lp < p.max_pages ? bt[lp] : -1;
      if (phys >= 0 && phys < p.num_pages)
        row = phys * P + (key - lp * P);
      else if (p.err)
        atomicOr(p.err, 1u << kErrTreeBadPage);
    }
#pragma unroll
    for (int c = 0; c < C::NCHUNK; ++c)
      tma_load_3d(dst + c * C::CHUNK_BYTES + r0 * 128, map, bar, c * 64, s.hk, row);
  }
}

// The low n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

template <int D, bool BF16, bool SOFTCAP>
__global__ void __launch_bounds__(TreeCfg<D>::THREADS, 1)
    attn_tree_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (no room at d = 128 to round the base up by hand: dynamic shared memory
  // starts at the window's 1024-byte base, and a launch where it does not ends
  // here with an error)
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, 1u << kErrTreeTeardown);
    return;
  }
  TreeSmem<C>& sm = *reinterpret_cast<TreeSmem<C>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool pair = p.two_tiles != 0;        // one query tile per warpgroup
  const int nq = pair ? 2 : 1;               // Q buffers
  const int ns = C::NBUF - nq;               // ring slots

  // This CTA's part of the line.
  const long long line = tree_total(p, sm.scan) * p.units;
  const int G = tree_ctas(p, line), cta = blockIdx.x;
  if (cta >= G) return;
  TreeWalk walk;
  {
    const long long x0 = line * cta / G, x1 = line * (cta + 1) / G;
    long long cum;
    tree_locate(p, x0, sm.scan, walk.b, cum);
    const int slots = tree_seq(p, walk.b).slots;
    const long long off = x0 - cum * p.units;
    walk.u = static_cast<int>(off / slots);
    walk.k = static_cast<int>(off - static_cast<long long>(walk.u) * slots);
    walk.rem = static_cast<int>(x1 - x0);
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBUF; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_half[t], 128);
      mbar_init(&sm.p_full[t], 128);
      mbar_init(&sm.o_final[t], 1);
    }
    mbar_init(&sm.o_free, 256);
    mbar_init(&sm.xch, 256);
    mbar_init(&sm.xread, 256);
    mbar_init(&sm.teardown, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&sm.tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const Waiter w{globaltimer_ns() + p.timeout_ns, &sm.abort_flag, p.err};
  TreeSeg s;
  bool first = true;

  if (warp >= 8) {
    setmaxnreg_dec<C::OTHER_REGS>();
    if (warp == 8 && lane == 0) {
      // ========================= TMA producer ================================
      tma_prefetch_desc(&p.tm_q);
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
      int seg = 0, item = 0;
      bool ok = true;
      for (; ok && tree_next(p, walk, s, first); first = false) {
        if (s.n == 0) continue;
        // Q goes out behind the segment's first K tile (the CTA's first one
        // before it): its buffer is free once the previous segment's last S is
        // done, which that K tile does not have to wait for.
        const int q_at = seg == 0 ? 0 : 1;
        for (int i = 0; ok && i < 2 * s.n; ++i, ++item) {
          if (i == q_at) {
            if (seg > 0 && !(ok = w.wait(&sm.q_empty, (seg - 1) & 1, kErrTreeWait))) break;
            const bool second = pair && s.m0 + p.qpt < p.T;
            mbar_arrive_expect_tx(&sm.q_full, (second ? 2 : 1) * p.qpt * p.g * D * 2);
            for (int t = 0; t < (second ? 2 : 1); ++t)
#pragma unroll
              for (int c = 0; c < C::NCHUNK; ++c)
                tma_load_5d(sm.buf[t] + c * C::CHUNK_BYTES, &p.tm_q, &sm.q_full, c * 64, 0, s.hk,
                            s.m0 + t * p.qpt, s.b);
            ++seg;
          }
          // item -> K or V of which tile
          bool is_v;
          int tile;
          if (i == 0) { tile = 0; is_v = false; }
          else if (i == 2 * s.n - 1) { tile = s.n - 1; is_v = true; }
          else if (i & 1) { tile = (i + 1) / 2; is_v = false; }
          else { tile = i / 2 - 1; is_v = true; }
          const int slot = item % ns;
          if (!(ok = w.wait(&sm.empty[slot], ((item / ns) & 1) ^ 1, kErrTreeWait))) break;
          mbar_arrive_expect_tx(&sm.full[slot], C::TILE_BYTES);
          tree_load_tile<C>(p, s, tree_tile(s.q, s.k0 + tile), is_v ? &p.tm_v : &p.tm_k, sm.buf[nq + slot],
                            &sm.full[slot]);
        }
      }
      if (w.aborted()) {
        // Every copy in flight lands before shared memory goes.
        const uint64_t dl = globaltimer_ns() + 50000000ull;
        if (seg > 0) wait_raw(&sm.q_full, (seg - 1) & 1, dl);
        for (int i = max(0, item - ns); i < item; ++i) wait_raw(&sm.full[i % ns], (i / ns) & 1, dl);
      }
    } else if (warp == 9) {
      // ========================= MMA issuer (whole warp) =====================
      const uint32_t lead = elect_one() ? 1u : 0u;
      constexpr uint32_t idesc_s = idesc_f16_f32(BF16, 128, C::BN, false, false);
      constexpr uint32_t idesc_o = idesc_f16_f32(BF16, 128, D, false, true);
      const uint64_t kdesc0 = sdesc_sw128(smem_u32(sm.buf[0]), 16, 1024);
      const uint64_t vdesc0 = sdesc_sw128(smem_u32(sm.buf[0]), C::CHUNK_BYTES, 1024);
      constexpr uint32_t kTileDesc = C::TILE_BYTES >> 4;
      int seg = 0, item0 = 0;
      uint32_t pph = 0;  // bit t: phase of tile t's next P
      bool ok = true;
      auto slot_of = [&](int it) { return (item0 + it) % ns; };
      auto wait_item = [&](int it) {
        return w.wait(&sm.full[slot_of(it)], ((item0 + it) / ns) & 1, kErrTreeWait);
      };
      auto issue_s = [&](int t, int i) {  // S_t = Q K_i^T
        const uint64_t qd = kdesc0 + static_cast<uint64_t>((pair ? t : 0) * kTileDesc);
        const uint64_t kd = kdesc0 + static_cast<uint64_t>((nq + slot_of(tree_k_item(i))) * kTileDesc);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * C::CHUNK_BYTES + (k & 3) * 32) >> 4;
          umma_ss_warp(tmem + C::tm_s(t), qd + off, kd + off, idesc_s, k > 0 ? 1u : 0u, lead);
        }
        umma_commit_warp(&sm.s_full[t], lead);
      };
      auto issue_pv = [&](int t, int slot, bool acc, int k0, int k1) {  // O_t (+)= P_t V
        const uint64_t vd = vdesc0 + static_cast<uint64_t>((nq + slot) * kTileDesc);
#pragma unroll
        for (int k = k0; k < k1; ++k)
          umma_ts_warp(tmem + C::tm_o(t), tmem + C::tm_s(t) + k * 8, vd + ((k * 16 * 128) >> 4), idesc_o,
                       (acc || k > 0) ? 1u : 0u, lead);
      };
      for (; ok && tree_next(p, walk, s, first); first = false) {
        if (s.n == 0) continue;
        const int n = s.n;
        const int live = pair ? (s.m0 + p.qpt < p.T ? 2 : 1) : min(n, 2);  // query tiles / streams in use
        if (!(ok = w.wait(&sm.q_full, seg & 1, kErrTreeWait))) break;
        // First S of each tile (alternate K tiles, or the same one).
        for (int t = 0; ok && t < live; ++t) {
          const int i = pair ? 0 : t;
          if (!(ok = wait_item(tree_k_item(i)))) break;
          tc_fence_after();
          issue_s(t, i);
          if (!pair || t == live - 1) umma_commit_warp(&sm.empty[slot_of(tree_k_item(i))], lead);
        }
        if (!ok) break;
        if (pair ? n == 1 : n <= 2) umma_commit_warp(&sm.q_empty, lead);  // no later S
        for (int i = 0; ok && i < n; ++i) {
          const int vslot = slot_of(tree_v_item(i, n));
          if (!(ok = wait_item(tree_v_item(i, n)))) break;
          {
            // Rows of the last page behind the sequence's end may hold anything,
            // and 0 * NaN in P.V is not 0: zero them.
            const int rows = s.q.L - tree_tile(s.q, s.k0 + i) * C::BN;
            if (rows < C::BN && rows % p.page_size != 0) {
              const int end = min(C::BN, (rows + p.page_size - 1) / p.page_size * p.page_size);
              for (int e = lane; e < (end - rows) * C::NCHUNK * 8; e += 32) {
                const int row = rows + e / (C::NCHUNK * 8), c = (e >> 3) % C::NCHUNK;
                *reinterpret_cast<uint4*>(sm.buf[nq + vslot] + c * C::CHUNK_BYTES + row * 128 + (e & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          const int step = pair ? 1 : 2;         // K tiles to this tile's next S
          const bool more = i + step < n;
          for (int t = pair ? 0 : (i & 1); ok && t < (pair ? live : (i & 1) + 1); ++t) {
            if (!(ok = w.wait(&sm.p_half[t], (pph >> t) & 1, kErrTreeWait))) break;
            const bool fresh = i < step;         // the tile's first P.V of the segment
            // O is free once the previous segment's epilogue has read it.
            if (fresh && seg > 0 && !(ok = w.wait(&sm.o_free, (seg - 1) & 1, kErrTreeWait))) break;
            tc_fence_after();
            issue_pv(t, vslot, !fresh, 0, C::BN / 32);
            if (!(ok = w.wait(&sm.p_full[t], (pph >> t) & 1, kErrTreeWait))) break;
            tc_fence_after();
            issue_pv(t, vslot, true, C::BN / 32, C::BN / 16);
            pph ^= 1u << t;
            if (!more) {
              umma_commit_warp(&sm.o_final[t], lead);
            } else {
              if (!(ok = wait_item(tree_k_item(i + step)))) break;
              issue_s(t, i + step);
            }
          }
          if (!ok) break;
          umma_commit_warp(&sm.empty[vslot], lead);
          if (more) {
            umma_commit_warp(&sm.empty[slot_of(tree_k_item(i + step))], lead);
            if (i + step == n - 1) umma_commit_warp(&sm.q_empty, lead);  // the segment's last S
          }
        }
        item0 += 2 * n;
        ++seg;
      }
      umma_commit_warp(&sm.teardown, lead);
      if (!wait_raw(&sm.teardown, 0, globaltimer_ns() + 50000000ull) && p.err)
        atomicOr(p.err, 1u << kErrTreeTeardown);
    }
  } else {
    setmaxnreg_inc<C::SOFT_REGS>();
    // ========================= softmax and epilogue ==========================
    const int t = warp >> 2;                    // query tile, or K/V stream
    const int r = (warp & 3) * 32 + lane;       // row == tensor-memory lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + C::tm_s(t) + lane_base;
    const int rq = r / p.g, hg = r - rq * p.g;  // query within the tile, head within the group
    int pc = 0, seg = 0;
    uint32_t oph = 0;  // bit i: phase of tile i's next final O
    bool ok = true;
    for (; ok && tree_next(p, walk, s, first); first = false) {
      const int n = s.n;
      const int live = pair ? (s.m0 + p.qpt < p.T ? 2 : 1) : min(n, 2);
      const int qi = s.m0 + (pair ? t * p.qpt : 0) + rq;
      const bool row_in = rq < p.qpt && qi < p.T;       // this thread has a row to write
      const bool row_live = row_in && qi < s.q.n;       // ... that sees anything
      const int hq = s.hk * p.g + hg;
      const int nt = t < live ? (pair ? n : (n + 1 - t) / 2) : 0;
      float m_use = -INFINITY, l = 0.0f;
      int lo = 0;  // lowest prefix key the window leaves
      if (p.win_left >= 0 && row_live) {
        const int depth = p.tree_depth != nullptr ? p.tree_depth[s.b * p.T + qi] : 0;
        lo = s.q.base + max(0, min(depth, s.q.n - 1)) - p.win_left;
      }
      const uint32_t* bits = p.tree_mask + (static_cast<int64_t>(s.b) * p.T + (row_live ? qi : 0)) * p.words;
      for (int j = 0; j < nt; ++j) {
        ok = __all_sync(0xffffffffu, w.wait(&sm.s_full[t], pc & 1, kErrTreeWait));
        if (!ok) break;
        ++pc;
        tc_fence_after();
        const int j0 = tree_tile(s.q, s.k0 + (pair ? j : 2 * j + t)) * C::BN;
        const bool masked = j0 + C::BN > s.q.base ||
                            (p.win_left >= 0 && j0 < s.q.base + s.q.n - p.win_left);
        uint32_t sr[C::BN];
        float raw_max = -INFINITY;
        if constexpr (!SOFTCAP) {
          uint32_t m4[4];
#pragma unroll
          for (int qq = 0; qq < 4; ++qq)
            tmem_ld32_max(tS + 32 * qq, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * qq]),
                          *reinterpret_cast<float*>(&m4[qq]));
          tmem_ld_wait();
          reg_fence(sr);
          reg_fence(m4);
          raw_max = fmaxf(fmax3(__uint_as_float(m4[0]), __uint_as_float(m4[1]), __uint_as_float(m4[2])),
                          __uint_as_float(m4[3]));
        } else {
#pragma unroll
          for (int qq = 0; qq < 4; ++qq)
            tmem_ld32(tS + 32 * qq, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * qq]));
          tmem_ld_wait();
          reg_fence(sr);
        }
        float* x = reinterpret_cast<float*>(sr);
        if constexpr (SOFTCAP) softcap_r_n<C::BN>(x, p.scale * p.softcap_inv);
        const float a_coef = SOFTCAP ? -2.0f * p.softcap * kLog2e : p.scale_log2;
        const float b_coef = SOFTCAP ? p.softcap * kLog2e : 0.0f;
        if (masked) {
          uint32_t vis[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k0 = j0 + 32 * c, sh = k0 - s.q.base;
            uint32_t pre = low_bits(-sh);  // keys before the drafted nodes
            if (p.win_left >= 0) pre &= ~low_bits(lo - k0) | low_bits(p.sink_tokens - k0);
            uint32_t node = 0;
            if (sh > -32 && sh < s.q.n) {
              const int wd = sh >> 5, bit = sh & 31;  // word -1 (none) below the first node
              const uint32_t w0 = wd >= 0 ? bits[wd] : 0u;
              const uint32_t w1 = bit != 0 && wd + 1 < p.words ? bits[wd + 1] : 0u;
              node = __funnelshift_r(w0, w1, bit) & low_bits(s.q.L - k0);
            }
            vis[c] = row_live ? pre | node : 0u;
          }
          constexpr float kDrop = SOFTCAP ? INFINITY : -INFINITY;
#pragma unroll
          for (int c = 0; c < C::BN; ++c) x[c] = (vis[c >> 5] >> (c & 31)) & 1u ? x[c] : kDrop;
        }
        float m_cand;
        if constexpr (SOFTCAP) m_cand = fmaf(min_n<C::BN>(x), a_coef, b_coef);
        else m_cand = (masked ? max_n<C::BN>(x) : raw_max) * a_coef;
        const float m_new = fmaxf(m_use, m_cand);
        float alpha = 1.0f;
        if (m_new - m_use > 8.0f) {  // false when both are -inf
          alpha = ex2_approx(m_use - m_new);
          m_use = m_new;
        }
        const float msub = m_use == -INFINITY ? 0.0f : m_use;
        uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pk[C::BN / 2];
        const uint64_t a2 = f2_pack(a_coef, a_coef), b2 = f2_pack(b_coef - msub, b_coef - msub);
        exp_pack_row<BF16, C::BN / 4>(x, a2, b2, pk, acc2);
        tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        // The tile's previous P.V was committed with this S: O can be rescaled.
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
          const uint32_t tO = tmem + C::tm_o(t) + lane_base;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t ov[32];
            tmem_ld32(tO + c, ov);
            tmem_ld_wait();
            reg_fence(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(tO + c, ov);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.p_half[t]);
        exp_pack_row<BF16, C::BN / 4>(x + C::BN / 2, a2, b2, pk + C::BN / 4, acc2);
        tmem_st32(tS + C::BN / 4, *reinterpret_cast<uint32_t(*)[32]>(&pk[C::BN / 4]));
        float r0, r1;
        f2_unpack(f2_add(f2_add(acc2[0], acc2[1]), f2_add(acc2[2], acc2[3])), r0, r1);
        l = l * alpha + (r0 + r1);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.p_full[t]);
      }
      if (!ok) break;

      // ---- epilogue.  With two query tiles each warpgroup owns its rows; with
      // two streams both hold parts of the same rows: they exchange (m, l) and
      // each merges half of the columns.
      float a0 = 1.0f, a1 = 0.0f, m = m_use;  // weights of the two streams' O
      if (!row_live) l = 0.0f, m = -INFINITY;
      if (!pair && n > 0) {
        // (the other warpgroup has read the previous segment's pair)
        if (seg > 0) ok = __all_sync(0xffffffffu, w.wait(&sm.xread, (seg - 1) & 1, kErrTreeWait));
        if (!ok) break;
        sm.x[t][r] = make_float2(m, l);
        mbar_arrive(&sm.xch);
        ok = __all_sync(0xffffffffu, w.wait(&sm.xch, seg & 1, kErrTreeWait));
        if (!ok) break;
        const float2 e0 = sm.x[0][r], e1 = sm.x[1][r];
        mbar_arrive(&sm.xread);
        m = fmaxf(e0.x, e1.x);
        const float ms = m == -INFINITY ? 0.0f : m;
        a0 = ex2_approx(e0.x - ms);
        a1 = ex2_approx(e1.x - ms);
        l = e0.y * a0 + e1.y * a1;
      }
      const bool use0 = pair ? (t < live && n > 0) : n > 0, use1 = !pair && n > 1;
      if (use0) {
        const int tt = pair ? t : 0;
        ok = __all_sync(0xffffffffu, w.wait(&sm.o_final[tt], (oph >> tt) & 1, kErrTreeWait));
        if (!ok) break;
      }
      if (use1) {
        ok = __all_sync(0xffffffffu, w.wait(&sm.o_final[1], oph >> 1, kErrTreeWait));
        if (!ok) break;
      }
      if (n > 0) oph ^= live == 2 ? 3u : 1u;
      tc_fence_after();

      float scale0 = a0, scale1 = a1, lse = -INFINITY;
      if (s.whole) {
        const float ms = m == -INFINITY ? 0.0f : m;
        float mfin = ms, ltot = l, norm = l > 0.0f ? 1.0f / l : 0.0f;
        if (p.sink != nullptr && row_in) {
          const float sl = p.sink[hq] * kLog2e;
          if (l > 0.0f) {
            mfin = fmaxf(ms, sl);
            const float a = ex2_approx(ms - mfin);
            ltot = l * a + ex2_approx(sl - mfin);
            norm = a / ltot;
          } else {
            mfin = sl;
            ltot = 1.0f;
          }
        }
        if (ltot > 0.0f) lse = (mfin + __log2f(ltot)) * kLn2;
        scale0 *= norm;
        scale1 *= norm;
      }
      const bool zero = !(l > 0.0f);  // nothing seen: O is 0 whatever the accumulator holds
      const int slot = cta * 2 + (s.first ? 0 : 1);
      const int prow = (pair ? t * 128 : 0) + r;                     // row of the piece
      const int prows = pair ? 256 : 128;
      float* part = p.o_part + static_cast<int64_t>(slot) * prows * D;
      T* out = reinterpret_cast<T*>(p.o) + ((static_cast<int64_t>(s.b) * p.T + qi) * p.Hq + hq) * D;
      const int c_beg = pair ? 0 : t * (D / 2), c_end = pair ? D : c_beg + D / 2;
      const bool writes = pair ? t < live || n == 0 : true;
      if (writes) {
        for (int c = c_beg; c < c_end; c += 32) {
          uint32_t o0[32], o1[32];
          if (use0) {
            tmem_ld32(tmem + C::tm_o(pair ? t : 0) + lane_base + c, o0);
            if (use1) tmem_ld32(tmem + C::tm_o(1) + lane_base + c, o1);
            tmem_ld_wait();
            reg_fence(o0);
            if (use1) reg_fence(o1);
          }
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] = 0.0f;
            if (use0 && !zero) v[i] = __uint_as_float(o0[i]) * scale0;
            if (use1 && !zero) v[i] = fmaf(__uint_as_float(o1[i]), scale1, v[i]);
          }
          if (row_in && s.whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w4[e] = BF16 ? pack_bf16(v[i + 2 * e], v[i + 2 * e + 1]) : pack_f16(v[i + 2 * e], v[i + 2 * e + 1]);
              *reinterpret_cast<uint4*>(out + c + i) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
          } else if (row_in) {
            // [D / 4][rows][4]: a warp's 32 rows are one 512-byte line.
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(part + (static_cast<int64_t>((c + i) / 4) * prows + prow) * 4) =
                  make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
          __syncwarp();
        }
        if (row_in && c_beg == 0) {
          if (s.whole) {
            if (p.lse != nullptr) p.lse[(static_cast<int64_t>(s.b) * p.Hq + hq) * p.T + qi] = lse;
          } else {
            p.ml_part[static_cast<int64_t>(slot) * prows + prow] = make_float2(zero ? -INFINITY : m, l);
          }
        }
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&sm.o_free);
        ++seg;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// Merges the pieces of every unit that was cut: block x handles the unit that
// holds the first tile of CTA x's range, if that tile lies inside the unit and
// no earlier CTA's first tile does; blockIdx.y picks 32 columns.  Thread = row.
//   M = max m_i, O = sum 2^(m_i - M) O_i / (sum 2^(m_i - M) l_i [+ 2^(sink - M)])
template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_tree_merge_kernel(const __grid_constant__ TreeParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  __shared__ long long scan[16];
  const long long line = tree_total(p, scan) * p.units;
  const int G = tree_ctas(p, line), c = blockIdx.x;
  if (c == 0 || c >= G) return;
  const long long x = line * c / G;
  int b;
  long long cum;
  tree_locate(p, x, scan, b, cum);
  const TreeSeq q = tree_seq(p, b);
  const long long off = x - cum * p.units;
  const int u = static_cast<int>(off / q.slots);
  const long long x0 = cum * p.units + static_cast<long long>(u) * q.slots, x1 = x0 + q.slots;
  // The CTAs whose ranges meet the unit; this block acts for the first inside it.
  const int c0 = static_cast<int>(((x0 + 1) * G - 1) / line), c1 = static_cast<int>((x1 * G - 1) / line);
  if (x == x0 || c != c0 + 1) return;
  const int rb = u / p.Hkv, hk = u - rb * p.Hkv;
  const int prows = p.two_tiles ? 256 : 128;
  const int row = threadIdx.x;  // blockDim.x == prows
  const int t = row >> 7, r = row & 127;
  const int rq = r / p.g, hg = r - rq * p.g;
  const int qi = rb * (p.two_tiles ? 2 : 1) * p.qpt + t * p.qpt + rq;
  if (rq >= p.qpt || qi >= p.T) return;
  const int hq = hk * p.g + hg;
  const float sl = p.sink != nullptr ? p.sink[hq] * kLog2e : -INFINITY;
  auto piece = [&](int i) {  // workspace piece of CTA i's part
    return static_cast<int64_t>(i) * 2 + (line * i / G >= x0 ? 0 : 1);
  };
  float M = sl;
  for (int i = c0; i <= c1; ++i) M = fmaxf(M, p.ml_part[piece(i) * prows + row].x);
  const float ms = M == -INFINITY ? 0.0f : M;
  float z = p.sink != nullptr ? ex2_approx(sl - ms) : 0.0f;
  float acc[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = 0.0f;
  const int col = blockIdx.y * 32;
  for (int i = c0; i <= c1; ++i) {
    const float2 e = p.ml_part[piece(i) * prows + row];
    const float wgt = ex2_approx(e.x - ms);
    z = fmaf(e.y, wgt, z);
    const float* part = p.o_part + piece(i) * prows * D;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float4 v = *reinterpret_cast<const float4*>(part + (static_cast<int64_t>((col + k) / 4) * prows + row) * 4);
      acc[k] = fmaf(v.x, wgt, acc[k]);
      acc[k + 1] = fmaf(v.y, wgt, acc[k + 1]);
      acc[k + 2] = fmaf(v.z, wgt, acc[k + 2]);
      acc[k + 3] = fmaf(v.w, wgt, acc[k + 3]);
    }
  }
  const float norm = z > 0.0f ? 1.0f / z : 0.0f;
  T* out = reinterpret_cast<T*>(p.o) + ((static_cast<int64_t>(b) * p.T + qi) * p.Hq + hq) * D + col;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    uint32_t w4[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = acc[i + 2 * e] * norm, hi = acc[i + 2 * e + 1] * norm;
      w4[e] = BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
    }
    *reinterpret_cast<uint4*>(out + i) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
  }
  if (col == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.T + qi] = z > 0.0f ? (ms + __log2f(z)) * kLn2 : -INFINITY;
}

template <int D, bool BF16, bool SOFTCAP>
static cudaError_t launch_tree_t(const TreeParams& p, cudaStream_t stream) {
  using C = TreeCfg<D>;
  auto kern = attn_tree_kernel<D, BF16, SOFTCAP>;
  const int smem = static_cast<int>(sizeof(TreeSmem<C>));
  static_assert(sizeof(TreeSmem<C>) <= 227 * 1024, "shared memory per block");
  // setmaxnreg.inc draws on what the block was launched with: refuse to launch
  // a build whose launch count is not the one the split assumes.
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != C::LAUNCH_REGS) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<p.grid, C::THREADS, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attn_tree_merge_kernel<D, BF16><<<dim3(p.grid, D / 32), p.two_tiles ? 256 : 128, 0, stream>>>(p);
  return cudaGetLastError();
}

template <>
cudaError_t launch_tree_d<ATTN_TREE_D>(const TreeParams& p, bool bf16, bool softcap, cudaStream_t stream) {
  if (bf16) return softcap ? launch_tree_t<ATTN_TREE_D, true, true>(p, stream)
                           : launch_tree_t<ATTN_TREE_D, true, false>(p, stream);
  return softcap ? launch_tree_t<ATTN_TREE_D, false, true>(p, stream)
                 : launch_tree_t<ATTN_TREE_D, false, false>(p, stream);
}

}  // namespace attn
