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
//    block, kv head) units form one line, each unit preceded by unit_cost
//    slots that stand for its start and epilogue, and CTA c takes the slots
//    [c T / G, (c + 1) T / G) of it, wherever sequence ends fall: every SM
//    gets the same amount of work for any mix of lengths.  The lengths live
//    on the device, so each CTA finds its place by a scan.  A unit that
//    ends up on one CTA is finished there; of a unit cut in pieces each CTA
//    writes (m, l, unnormalised O) to the workspace (at most two pieces per
//    CTA: its first and its last) and a second kernel merges them.
//  * where there are enough units to balance the CTAs without cuts (two to
//    sixteen per CTA), whole units are dealt out instead, longest first in
//    snake order, if the longest hand is not much above the mean (every CTA
//    works that out alike from the lengths).
//  * up to 128 rows per unit, one query tile is not enough to hide the chain
//    S -> softmax -> P.V behind the loads: the two softmax warpgroups then take
//    alternate K/V tiles of the unit, each with its own running maximum, sum
//    and O accumulator, merged from tensor memory at the unit's end.  Above
//    128 rows they take one query tile each and share every K/V tile.
//  * K and V tiles pass through one ring of shared-memory slots in consumption
//    order (K0, K1, V0, K2, V1, ... for two streams, K0, V0, K1, V1, ... for two
//    query tiles); what Q does not take of shared memory is ring (d = 128: 6
//    slots of 32 KB, or 5 beside two query tiles).
//  * without masks (tree_mask NULL) the T queries are the sequence's last tokens, a
//    plain causal chunk: single-token decode with a window and first tokens runs
//    here where there are enough units (attn_fwd_paged).
//  * only the tiles that hold drafted nodes, the sequence's end or a window's
//    edge are masked, from a 128-bit visibility word per row.
#pragma once
#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "softmax.cuh"

#include <atomic>
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
  uint64_t s_full[2], p_half[2], p_full[2], o_final[2], o_free[2], xch, xread;
  uint64_t teardown;
  float2 x[2][128];     // (m, l) of a row, per warpgroup
  int scan[16];
  int4 desc[4][3];      // segments on their way from the producer to the other roles
  uint64_t desc_full[4], desc_empty[4];
  uint8_t order[256];   // unit mode: the sequences, most tiles first
  uint32_t tmem_base;
  int abort_flag;
};

// What the kernel needs to know of one sequence.
struct TreeSeq {
  int L, base, n;     // keys, keys before the drafted nodes, nodes
  int nkeep, gap;     // tile of step k: k < nkeep ? k : k + gap
  int tiles;          // K/V tiles with a visible key
  int slots;          // its share of the work line per unit: tiles + unit_cost
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
  s.slots = s.tiles + p.unit_cost;
  return s;
}

// The line of tile slots in equal parts: CTA c of G takes [start(c), start(c + 1)).
struct TreeLine {
  int len, G, q, rem;
  __device__ __forceinline__ int start(int c) const { return c * q + min(c, rem); }
  __device__ __forceinline__ int cta_of(int x) const {
    const int big = rem * (q + 1);
    return x < big ? x / (q + 1) : rem + (x - big) / q;
  }
};

__device__ __forceinline__ TreeLine tree_line(const TreeParams& p, int total) {
  TreeLine n;
  n.len = total * p.units;
  n.G = min((n.len + p.min_share - 1) / p.min_share, p.grid);
  n.q = n.len / n.G;
  n.rem = n.len - n.q * n.G;
  return n;
}

// The line, and the sequence whose slots hold this CTA's first one: b, with
// cum slots per unit before it.  A block-wide scan over the sequences'
// lengths; every thread returns the same values (b = -1: nothing for this
// CTA).  Up to blockDim sequences it takes one pass.  At most 14 warps;
// scratch: 16 ints.
__device__ inline TreeLine tree_place(const TreeParams& p, int* scratch, int& b_out, int& cum_out) {
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool one = p.B <= static_cast<int>(blockDim.x);
  TreeLine line{};
  int total = 0, x = 0;
  if (!one) {
    int v = 0;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) v += tree_seq(p, b).slots;
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    for (int i = 0; i < warps; ++i) total += scratch[i];
    line = tree_line(p, total);
    x = line.start(blockIdx.x);
  }
  if (threadIdx.x == 0) scratch[14] = -1;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const int n = b < p.B ? tree_seq(p, b).slots : 0;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();  // the previous sums have been read
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int pre = before, all = before;
    for (int i = 0; i < warps; ++i) {
      if (i < warp) pre += scratch[i];
      all += scratch[i];
    }
    if (one) {
      line = tree_line(p, all);
      x = line.start(blockIdx.x);
    }
    const int lo = (pre + inc - n) * p.units;
    if (static_cast<int>(blockIdx.x) < line.G && b < p.B && lo <= x && x - lo < n * p.units) {
      scratch[14] = b;
      scratch[15] = pre + inc - n;
    }
    before = all;
  }
  __syncthreads();
  b_out = scratch[14];
  cum_out = scratch[15];
  return line;
}

// Unit mode: hand of CTA c is items c, 2G - 1 - c, 2G + c, ... of the B * units
// units, sequences with most tiles first.
__device__ __forceinline__ int tree_item(int G, int c, int round) {
  return round * G + ((round & 1) ? G - 1 - c : c);
}

// Decides for the whole grid between the line and unit mode, and leaves the
// sequences' order in `order`.  The limit: a cut costs a CTA another start and
// epilogue (2 unit_cost) and the merge kernel about 8 tiles' time; the snake's
// uneven hands cost up to a sixteenth there.  cost: 256 ints of scratch.
__device__ inline bool tree_unit_mode(const TreeParams& p, const TreeLine& line, int* scratch, int* cost,
                                      uint8_t* order) {
  const int N = p.B * p.units, G = gridDim.x, warp = threadIdx.x >> 5;
  const bool always = p.o_part == nullptr;  // no workspace for pieces: the host has checked the counts
  if (p.B > 256 || N < 2 * G || (N > 16 * G && !always)) return always;
  const int b = threadIdx.x;
  if (b < p.B) cost[b] = tree_seq(p, b).slots;
  __syncthreads();
  if (b < p.B) {
    const int mine = cost[b];
    int rank = 0;
    for (int j = 0; j < p.B; ++j) rank += cost[j] > mine || (cost[j] == mine && j < b);
    order[rank] = static_cast<uint8_t>(b);
  }
  __syncthreads();
  int hand = 0;
  if (b < G)
    for (int k = 0, i; (i = tree_item(G, b, k)) < N; ++k) hand += cost[order[i / p.units]];
  hand = __reduce_max_sync(0xffffffffu, hand);
  if ((threadIdx.x & 31) == 0) scratch[warp] = hand;
  __syncthreads();
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) hand = max(hand, scratch[i]);
  fence_proxy_async_smem();  // `cost` lies where the first copies will land
  __syncthreads();
  return always || hand <= line.q + line.q / 16 + 2 * p.unit_cost + 8;
}

// A CTA's walk along the line, one segment (a run of tiles of one unit) at a time.
struct TreeWalk {
  int b, u, k;    // next sequence, unit within it, slot; unit mode: -2, -, round
  int rem;        // slots left
};
struct TreeSeg {
  TreeSeq q;
  int b, hk, m0;    // sequence, kv head, first query
  int k0, n;        // tile steps [k0, k0 + n) of the unit
  bool whole;       // the unit's only segment
};

// (A segment of no tiles is a part of a unit's leading slots, with nothing to
// do, unless the unit has no tile at all: its first segment is then whole.)
__device__ __forceinline__ bool tree_next(const TreeParams& p, const uint8_t* order, TreeWalk& w, TreeSeg& s) {
  if (w.rem <= 0) return false;
  if (w.b == -2) {
    const int i = tree_item(gridDim.x, blockIdx.x, w.k);
    if (i >= p.B * p.units) return false;
    ++w.k;
    s.b = order[i / p.units];
    const int u = i % p.units, rb = u / p.Hkv;
    s.hk = u - rb * p.Hkv;
    s.m0 = rb * (p.two_tiles ? 2 : 1) * p.qpt;
    s.q = tree_seq(p, s.b);
    s.k0 = 0;
    s.n = s.q.tiles;
    s.whole = true;
    return true;
  }
  s.q = tree_seq(p, w.b);
  const int take = min(w.rem, s.q.slots - w.k);
  s.b = w.b;
  const int rb = w.u / p.Hkv;
  s.hk = w.u - rb * p.Hkv;
  s.m0 = rb * (p.two_tiles ? 2 : 1) * p.qpt;
  s.k0 = max(w.k - p.unit_cost, 0);
  s.n = max(w.k + take - p.unit_cost, 0) - s.k0;
  s.whole = s.n == s.q.tiles && (s.n > 0 || w.k == 0);
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

// Segments are worked out once, by the K producer, which runs ahead of the
// others, and handed on through shared memory (three 16-byte words): the
// softmax warps' time between two segments is all dependent scalar code, and
// the walk was a third of it.  n = -1 ends the walk.
__device__ __forceinline__ void tree_pack(const TreeSeg& s, int4 (&w)[3]) {
  w[0] = make_int4(s.b, s.hk, s.m0, s.n);
  w[1] = make_int4(s.k0, s.q.L, s.q.base, s.q.n);
  w[2] = make_int4(s.q.nkeep, s.q.gap, s.q.tiles, s.whole ? 1 : 0);
}
template <class C>
__device__ __forceinline__ void tree_read(const TreeSmem<C>& sm, int slot, TreeSeg& s) {
  const int4 a = sm.desc[slot][0], b = sm.desc[slot][1], c = sm.desc[slot][2];
  s.b = a.x, s.hk = a.y, s.m0 = a.z, s.n = a.w;
  s.k0 = b.x, s.q.L = b.y, s.q.base = b.z, s.q.n = b.w;
  s.q.nkeep = c.x, s.q.gap = c.y, s.q.tiles = c.z, s.whole = c.w != 0;
}
// The k-th segment is in its slot (false: a wait gave up).  Released when the
// warp needs it no more.
template <class C>
__device__ __forceinline__ bool tree_wait(TreeSmem<C>& sm, const Waiter& w, int k) {
  return __all_sync(0xffffffffu, w.wait(&sm.desc_full[k & 3], (k >> 2) & 1, kErrTreeWait));
}
template <class C>
__device__ __forceinline__ void tree_release(TreeSmem<C>& sm, int k) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.desc_empty[k & 3]);
}
template <class C>
__device__ __forceinline__ bool tree_take(TreeSmem<C>& sm, const Waiter& w, int& k, TreeSeg& s) {
  if (!tree_wait(sm, w, k)) return false;
  tree_read(sm, k & 3, s);
  tree_release(sm, k);
  ++k;
  return s.n >= 0;
}

__device__ __forceinline__ int tree_tile(const TreeSeq& q, int k) { return k < q.nkeep ? k : k + q.gap; }

// Pool row of page piece `lane` of a tile (box of min(page, 128) rows).  Pieces
// behind the sequence's end, without a visible key, or behind a bad table
// entry (an error) read one row past the pool: zeros.
template <class C>
__device__ __forceinline__ int tree_piece_row(const TreeParams& p, const TreeSeg& s, int tile, int lane) {
  const int br_log2 = min(p.page_log2, 7);
  const int key = tile * C::BN + (lane << br_log2);
  const int klo = p.win_left >= 0 ? max(0, s.q.base - p.win_left) : 0;
  const int none = p.num_pages << p.page_log2;
  if (lane >= (C::BN >> br_log2) || key >= s.q.L || (key + (1 << br_log2) <= klo && key >= p.sink_tokens))
    return none;
  const int lp = key >> p.page_log2;
  const int phys = lp < p.max_pages ? p.block_table[static_cast<int64_t>(s.b) * p.max_pages + lp] : -1;
  if (phys >= 0 && phys < p.num_pages) return (phys << p.page_log2) + (key & (p.page_size - 1));
  if (p.err) atomicOr(p.err, 1u << kErrTreeBadPage);
  return none;
}

// 4 x 4 transpose of 16-byte pieces within each quad of lanes: piece i of lane q
// becomes piece q of lane i.  w: four pieces of four words.  (Selects on both
// sides, no indexing by lane: that would put the array in local memory.)
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[16], int lane) {
  const bool hi2 = lane & 2, hi1 = lane & 1;
#pragma unroll
  for (int e = 0; e < 8; ++e) {  // pieces 0, 1 against 2, 3
    const uint32_t got = __shfl_xor_sync(0xffffffffu, hi2 ? w[e] : w[e + 8], 2);
    w[e] = hi2 ? got : w[e];
    w[e + 8] = hi2 ? w[e + 8] : got;
  }
#pragma unroll
  for (int h = 0; h < 16; h += 8)
#pragma unroll
    for (int e = h; e < h + 4; ++e) {  // pieces 0 against 1, 2 against 3
      const uint32_t got = __shfl_xor_sync(0xffffffffu, hi1 ? w[e] : w[e + 4], 1);
      w[e] = hi1 ? got : w[e];
      w[e + 4] = hi1 ? w[e + 4] : got;
    }
}

// pair: units of two query tiles, one per softmax warpgroup; else one tile and two
// streams of K/V tiles (see the top of the file).
template <int D, bool BF16, bool SOFTCAP, bool pair>
__global__ void __launch_bounds__(TreeCfg<D>::THREADS, 1)
    attn_tree_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (no room at d = 128 to round the base up by hand: dynamic shared memory
  // starts at the window's 1024-byte base, and a launch where it does not ends
  // here with an error, and nothing for the merge kernel to do)
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    pdl_wait();
    if (threadIdx.x == 0) {
      if (p.err) atomicOr(p.err, 1u << kErrTreeTeardown);
      if (p.o_part != nullptr) p.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    return;
  }
  TreeSmem<C>& sm = *reinterpret_cast<TreeSmem<C>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int nq = pair ? 2 : 1;           // Q buffers
  constexpr int ns = C::NBUF - nq;           // ring slots

  pdl_launch_dependents();  // the merge kernel may be set up; it waits for this grid's end
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
      mbar_init(&sm.o_free[t], pair ? 128 : 256);  // the threads that read the tile's O
    }
    mbar_init(&sm.xch, 256);
    mbar_init(&sm.xread, 256);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.desc_full[i], 1);
      mbar_init(&sm.desc_empty[i], 10);  // 8 softmax warps, the V producer, the MMA issuer
    }
    mbar_init(&sm.teardown, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == 9) {
    tmem_alloc(&sm.tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  // This CTA's part of the line.  (Up to here nothing was read that an earlier
  // kernel of the stream may still be writing.)
  pdl_wait();
  tc_fence_before();
  const int cta = blockIdx.x;
  TreeWalk walk;
  int cum;
  const TreeLine line = tree_place(p, sm.scan, walk.b, cum);  // (synchronises the block)
  const bool deal = tree_unit_mode(p, line, sm.scan, reinterpret_cast<int*>(sm.buf[0]), sm.order);
  tc_fence_after();
  if (deal) {
    walk = TreeWalk{-2, 0, 0, 1};
    if (threadIdx.x == 0 && p.o_part != nullptr) p.cut[cta] = make_int4(-1, 0, 0, 0);
  } else if (walk.b < 0) {
    walk.rem = 0;
    if (threadIdx.x == 0) p.cut[cta] = make_int4(-1, 0, 0, 0);
  } else {
    const int slots = tree_seq(p, walk.b).slots, x = line.start(cta);
    const int off = x - cum * p.units;
    walk.u = off / slots;
    walk.k = off - walk.u * slots;
    walk.rem = line.start(cta + 1) - x;
    if (threadIdx.x == 0) {
      // For the merge kernel: this CTA's first tile is inside a unit, and the
      // CTA before it holds the unit's tile 0.
      const int x0 = x - walk.k;
      const bool first_cut = walk.k > p.unit_cost && line.start(cta - 1) <= x0 + p.unit_cost;
      p.cut[cta] = first_cut ? make_int4(walk.b, walk.u, line.cta_of(x0 + slots - 1), 0)
                             : make_int4(-1, 0, 0, 0);
    }
  }
  const uint32_t tmem = sm.tmem_base;
  const Waiter w{globaltimer_ns() + p.timeout_ns, &sm.abort_flag, p.err};
  TreeSeg s;

  if (warp >= 8) {
    setmaxnreg_dec<C::OTHER_REGS>();
    if (warp == 8 || warp == 10) {
      // ========================= TMA producers (whole warps) =================
      // Warp 8 loads Q and the K tiles, warp 10 the V tiles, each into its items
      // of the one ring.  A tile is up to 8 page pieces x 2 column atoms: the
      // lanes look the pieces' pages up together, a tile ahead, and the warp
      // issues the boxes with a uniform row (measured at 16-token pages: one
      // lane doing both in turn needs 3400 cycles per K and V tile, the step
      // itself 2000).
      const bool v_warp = warp == 10;
      const CUtensorMap* map = v_warp ? &p.tm_v : &p.tm_k;
      const uint32_t lead = elect_one() ? 1u : 0u;
      const int br_log2 = min(p.page_log2, 7), pieces = C::BN >> br_log2;
      int seg = 0, armed = 0, slot = 0;  // slot: the ring slot of the segment's next item
      uint32_t eph = 1;                  // and the parity its release is waited with
      bool ok = true;
      // Items before this warp's next one that are the other warp's.
      auto skip = [&](int n) {
        slot += n;
        if (slot >= ns) slot -= ns, eph ^= 1;
      };
      auto load = [&](int row) {  // one tile into the current slot
        ok = __all_sync(0xffffffffu, w.wait(&sm.empty[slot], eph, kErrTreeWait));
        if (!ok) return;
        if (lead) mbar_arrive_expect_tx(&sm.full[slot], C::TILE_BYTES);
        __syncwarp();
        uint8_t* dst = sm.buf[nq + slot];
        for (int i = 0; i < pieces; ++i) {
          const int r = __shfl_sync(0xffffffffu, row, i);
#pragma unroll
          for (int c = 0; c < C::NCHUNK; ++c)
            tma_load_3d_warp(dst + c * C::CHUNK_BYTES + (i << (br_log2 + 7)), map, &sm.full[slot], c * 64, s.hk,
                             r, lead);
        }
        ++armed;
        skip(1);
      };
      int dk = 0;  // segments handed on or taken
      while (ok) {
        if (!v_warp) {
          s.n = -1;
          bool more;
          while ((more = tree_next(p, sm.order, walk, s)) && s.n == 0 && !s.whole) {
          }
          if (!more) s.n = -1;
          ok = __all_sync(0xffffffffu, w.wait(&sm.desc_empty[dk & 3], ((dk >> 2) & 1) ^ 1, kErrTreeWait));
          if (!ok) break;
          if (lane == 0) {
            int4 d[3];
            tree_pack(s, d);
            for (int i = 0; i < 3; ++i) sm.desc[dk & 3][i] = d[i];
            mbar_arrive(&sm.desc_full[dk & 3]);
          }
          __syncwarp();
          ++dk;
          if (!more) break;
        } else if (!tree_take(sm, w, dk, s)) {
          break;
        }
        const int n = __shfl_sync(0xffffffffu, s.n, 0);
        if (n == 0) continue;
        int row = tree_piece_row<C>(p, s, tree_tile(s.q, s.k0), lane);
        for (int i = 0; ok && i < n; ++i) {
          const int next = i + 1 < n ? tree_piece_row<C>(p, s, tree_tile(s.q, s.k0 + i + 1), lane) : 0;
          if (!v_warp) {
            // Q goes out behind the segment's first K tile (the CTA's first one
            // before it): its buffer is free once the previous segment's last S
            // is done, which that K tile does not have to wait for.
            for (int part = 0; ok && part < 2; ++part) {
              const bool q_part = seg == 0 ? part == 0 : part == 1;
              if (!q_part) {
                load(row);
                // pair: K_i V_i K_i+1; streams: K0 K1 V0 K2 V1 ... V_n-2 V_n-1
                if (ok) skip(pair ? 1 : i == 0 ? (n == 1 ? 1 : 0) : i == n - 1 ? 2 : 1);
              } else if (i == 0) {
                ok = seg == 0 || __all_sync(0xffffffffu, w.wait(&sm.q_empty, (seg - 1) & 1, kErrTreeWait));
                if (!ok) break;
                const int nt = pair && s.m0 + p.qpt < p.T ? 2 : 1;
                if (lead) {
                  mbar_arrive_expect_tx(&sm.q_full, nt * p.qpt * p.g * D * 2);
                  for (int t = 0; t < nt; ++t)
#pragma unroll
                    for (int c = 0; c < C::NCHUNK; ++c)
                      tma_load_5d(sm.buf[t] + c * C::CHUNK_BYTES, &p.tm_q, &sm.q_full, c * 64, 0, s.hk,
                                  s.m0 + t * p.qpt, s.b);
                }
                __syncwarp();
              }
            }
          } else {
            if (i == 0) skip(pair || n == 1 ? 1 : 2);
            load(row);
            if (ok) skip(pair ? (i + 1 < n ? 1 : 0) : i + 2 < n ? 1 : 0);
          }
          row = next;
        }
        ++seg;
      }
      if (w.aborted()) {
        // Every copy in flight lands before shared memory goes: each slot's
        // last armed phase completes when its bytes arrive (a slot never armed,
        // or armed by the other warp, is waited for at most until the limit).
        const uint64_t dl = globaltimer_ns() + 50000000ull;
        if (!v_warp && seg > 0) wait_raw(&sm.q_full, (seg - 1) & 1, dl);
        for (int i = 0; i < ns && armed > 0; ++i) wait_raw(&sm.full[i], i < slot ? eph ^ 1 : eph, dl);
      }
    } else if (warp == 9) {
      // ========================= MMA issuer (whole warp) =====================
      // The issue rate of this warp bounds the step (16 MMAs and 3 commits per
      // tile): tiles are compile-time constants here and the ring position is
      // a cursor, never a division (measured: 1400 cycles per tile's step with
      // run-time tiles and item % slots).
      const uint32_t lead = elect_one() ? 1u : 0u;
      constexpr uint32_t idesc_s = idesc_f16_f32(BF16, 128, C::BN, false, false);
      constexpr uint32_t idesc_o = idesc_f16_f32(BF16, 128, D, false, true);
      constexpr uint32_t kTileDesc = C::TILE_BYTES >> 4;
      const uint64_t qdesc0 = sdesc_sw128(smem_u32(sm.buf[0]), 16, 1024);
      const uint64_t qdesc1 = qdesc0 + (pair ? kTileDesc : 0);
      const uint64_t kdesc0 = sdesc_sw128(smem_u32(sm.buf[nq]), 16, 1024);
      const uint64_t vdesc0 = sdesc_sw128(smem_u32(sm.buf[nq]), C::CHUNK_BYTES, 1024);
      int seg = 0, cur = 0;          // ring slot of the next item
      uint32_t cph = 0;              // and its phase
      uint32_t pph0 = 0, pph1 = 0;   // phase of each tile's next P
      auto advance = [&]() {
        if (++cur == ns) cur = 0, cph ^= 1;
      };
      auto issue_s = [&](auto tc, int slot) {  // S_t = Q K^T
        constexpr int t = decltype(tc)::value;
        const uint64_t qd = t ? qdesc1 : qdesc0;
        const uint64_t kd = kdesc0 + static_cast<uint64_t>(slot * kTileDesc);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          constexpr uint32_t kIn = 32 >> 4;
          const uint32_t off = (k >> 2) * (C::CHUNK_BYTES >> 4) + (k & 3) * kIn;
          umma_ss_warp(tmem + C::tm_s(t), qd + off, kd + off, idesc_s, k > 0 ? 1u : 0u, lead);
        }
        umma_commit_warp(&sm.s_full[t], lead);
      };
      // P.V of tile t as its two halves arrive.  fresh: the tile's first of the
      // segment (O is free once the previous segment's epilogue has read it).
      auto issue_pv = [&](auto tc, int slot, bool fresh) -> bool {
        constexpr int t = decltype(tc)::value;
        uint32_t& ph = t ? pph1 : pph0;
        const uint64_t vd = vdesc0 + static_cast<uint64_t>(slot * kTileDesc);
        if (!w.wait(&sm.p_half[t], ph, kErrTreeWait)) return false;
        if (fresh && seg > 0 && !w.wait(&sm.o_free[t], (seg - 1) & 1, kErrTreeWait)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < C::BN / 32; ++k)
          umma_ts_warp(tmem + C::tm_o(t), tmem + C::tm_s(t) + k * 8, vd + ((k * 16 * 128) >> 4), idesc_o,
                       (k > 0 || !fresh) ? 1u : 0u, lead);
        if (!w.wait(&sm.p_full[t], ph, kErrTreeWait)) return false;
        ph ^= 1;
        tc_fence_after();
#pragma unroll
        for (int k = C::BN / 32; k < C::BN / 16; ++k)
          umma_ts_warp(tmem + C::tm_o(t), tmem + C::tm_s(t) + k * 8, vd + ((k * 16 * 128) >> 4), idesc_o, 1u,
                       lead);
        return true;
      };
      const std::integral_constant<int, 0> t0{};
      const std::integral_constant<int, 1> t1{};
      bool ok = true;
      int dk = 0;
      while (ok && tree_take(sm, w, dk, s)) {
        if (s.n == 0) continue;
        const int n = __shfl_sync(0xffffffffu, s.n, 0);
        const bool two = pair ? s.m0 + p.qpt < p.T : n > 1;  // both tiles in use
        const int tail = s.q.L & (C::BN - 1);  // rows of the sequence's last tile, if not full
        const int last = s.k0 + n == s.q.tiles && (tail & (p.page_size - 1)) != 0 ? n - 1 : -1;
        if (!(ok = w.wait(&sm.q_full, seg & 1, kErrTreeWait))) break;
        // First S of each tile: of K0, and of K1 where the tiles are streams.
        if (!(ok = w.wait(&sm.full[cur], cph, kErrTreeWait))) break;
        tc_fence_after();
        issue_s(t0, cur);
        if (pair) {
          if (two) issue_s(t1, cur);
          umma_commit_warp(&sm.empty[cur], lead);
          advance();
        } else {
          umma_commit_warp(&sm.empty[cur], lead);
          advance();
          if (two) {
            if (!(ok = w.wait(&sm.full[cur], cph, kErrTreeWait))) break;
            tc_fence_after();
            issue_s(t1, cur);
            umma_commit_warp(&sm.empty[cur], lead);
            advance();
          }
        }
        if (pair ? n == 1 : n <= 2) umma_commit_warp(&sm.q_empty, lead);  // no later S
        const int step = pair ? 1 : 2;  // K tiles from one S of a tile to its next
        for (int i = 0; i < n; ++i) {
          const int vs = cur;
          if (!(ok = w.wait(&sm.full[vs], cph, kErrTreeWait))) break;
          advance();
          if (i == last) {
            // Rows of the last page behind the sequence's end may hold anything,
            // and 0 * NaN in P.V is not 0: zero them.
            const int end = min(C::BN, (tail + p.page_size - 1) & ~(p.page_size - 1));
            for (int e = lane; e < (end - tail) * C::NCHUNK * 8; e += 32) {
              const int row = tail + e / (C::NCHUNK * 8), c = (e >> 3) % C::NCHUNK;
              *reinterpret_cast<uint4*>(sm.buf[nq + vs] + c * C::CHUNK_BYTES + row * 128 + (e & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          const bool more = i + step < n, fresh = i < step;
          const int ks = cur;  // K tile of the next S, behind V in the ring
          const uint32_t kph = cph;
          // One tile's part of the step: P.V, then its next S.
          auto part = [&](auto tc) -> bool {
            constexpr int t = decltype(tc)::value;
            if (!issue_pv(tc, vs, fresh)) return false;
            if (more) {
              if (!w.wait(&sm.full[ks], kph, kErrTreeWait)) return false;
              tc_fence_after();
              issue_s(tc, ks);
            } else {
              umma_commit_warp(&sm.o_final[t], lead);
            }
            return true;
          };
          if (pair) ok = part(t0) && (!two || part(t1));
          else ok = (i & 1) ? part(t1) : part(t0);
          if (!ok) break;
          umma_commit_warp(&sm.empty[vs], lead);
          if (more) {
            umma_commit_warp(&sm.empty[ks], lead);
            advance();
            if (i + step == n - 1) umma_commit_warp(&sm.q_empty, lead);  // the segment's last S
          }
        }
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
    // Division of a row by the group size, in two instructions (exact below
    // 128): the registers are better spent on scores than on keeping quotients.
    auto div_g = [&](int x) { return (x * p.g_magic) >> 16; };
    int pc = 0, seg = 0;
    uint32_t oph = 0;  // bit i: phase of tile i's next final O
    bool ok = true;
    // The scores take 128 of the 192 registers: of the segment only what the loop
    // over its tiles needs stays in registers, the rest is read again from shared
    // memory where a masked tile or the epilogue asks for it.
    auto rows_of = [&](const TreeSeg& e, int& qi, int& hq, bool& in) {  // this thread's row
      const int rq = div_g(r);
      qi = e.m0 + (pair ? t * p.qpt : 0) + rq;
      hq = e.hk * p.g + (r - rq * p.g);
      in = rq < p.qpt && qi < p.T;
    };
    // Whether the row may see anything: a node in use; in a chain, a position.
    auto sees = [&](const TreeSeg& e, int qi) {
      return p.tree_mask != nullptr ? qi < e.q.n : e.q.L - p.T + qi >= 0;
    };
    for (int dk = 0; ok; ++dk) {
      if (!(ok = tree_wait(sm, w, dk))) break;
      tree_read(sm, dk & 3, s);
      const int n = s.n;
      if (n < 0) break;
      const int live = pair ? (s.m0 + p.qpt < p.T ? 2 : 1) : min(n, 2);
      const int nt = t < live ? (pair ? n : (n + 1 - t) / 2) : 0;
      float m_use = -INFINITY, l = 0.0f;
      for (int j = 0; j < nt; ++j) {
        const int j0 = tree_tile(s.q, s.k0 + (pair ? j : 2 * j + t)) * C::BN;
        const bool masked = j0 + C::BN > s.q.base ||
                            (p.win_left >= 0 && j0 < s.q.base + s.q.n - p.win_left);
        // Which keys of a masked tile the row sees, worked out (and its mask
        // words fetched) while the tensor core computes the scores.
        uint32_t vis[4] = {0u, 0u, 0u, 0u};
        TreeSeg e;
        int qi, hq;
        bool row_live = false;
        if (masked) {
          tree_read(sm, dk & 3, e);
          rows_of(e, qi, hq, row_live);
          row_live = row_live && sees(e, qi);
        }
        if (row_live && p.tree_mask == nullptr) {
          // A chain: keys up to the query's own position, within the window.
          const int pos = e.q.L - p.T + qi, lo = p.win_left >= 0 ? pos - p.win_left : 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k0 = j0 + 32 * c;
            vis[c] = low_bits(pos + 1 - k0) & (~low_bits(lo - k0) | low_bits(p.sink_tokens - k0));
          }
        } else if (row_live) {
          const int64_t node_row = static_cast<int64_t>(e.b) * p.T + qi;
          const uint32_t* bits = p.tree_mask + node_row * p.words;
          const int sh0 = j0 - e.q.base;  // first column, counted from node 0
          const int wd = sh0 >> 5, bit = sh0 & 31;
          // (Ordinary loads here and of the depth: the kernel that writes them may
          // still run when this one starts, which the read-only path does not allow.)
          uint32_t wds[5];
#pragma unroll
          for (int c = 0; c < 5; ++c)
            wds[c] = wd + c >= 0 && wd + c < p.words ? bits[wd + c] : 0u;
          int lo = 0;  // lowest key before the nodes that the window leaves
          if (p.win_left >= 0)
            lo = e.q.base + max(0, min(p.tree_depth[node_row], e.q.n - 1)) - p.win_left;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k0 = j0 + 32 * c;
            uint32_t pre = low_bits(e.q.base - k0);  // keys before the nodes
            if (p.win_left >= 0) pre &= ~low_bits(lo - k0) | low_bits(p.sink_tokens - k0);
            vis[c] = pre | (__funnelshift_r(wds[c], wds[c + 1], bit) & low_bits(e.q.L - k0));
          }
        }
        ok = __all_sync(0xffffffffu, w.wait(&sm.s_full[t], pc & 1, kErrTreeWait));
        if (!ok) break;
        ++pc;
        tc_fence_after();
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
      tree_read(sm, dk & 3, s);
      int qi, hq;
      bool row_in;  // this thread has a row to write
      rows_of(s, qi, hq, row_in);
      const bool row_live = row_in && sees(s, qi);
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
      // Everything that does not need O comes before the wait for it.  (l is 0 where
      // the row has seen nothing, and NaN, which has to come out, where a score was:
      // hence comparisons with 0 and not l > 0.)
      float scale0 = a0, scale1 = a1, lse = -INFINITY;
      if (s.whole) {
        const float ms = m == -INFINITY ? 0.0f : m;
        float mfin = ms, ltot = l, norm = l != 0.0f ? rcp_approx(l) : 0.0f;
        if (p.sink != nullptr && row_in) {
          const float sl = p.sink[hq] * kLog2e;
          if (l != 0.0f) {
            mfin = fmaxf(ms, sl);
            const float a = ex2_approx(ms - mfin);
            ltot = l * a + ex2_approx(sl - mfin);
            norm = a * rcp_approx(ltot);
          } else {
            mfin = sl;
            ltot = 1.0f;
          }
        }
        if (ltot != 0.0f) lse = (mfin + __log2f(ltot)) * kLn2;
        scale0 *= norm;
        scale1 *= norm;
      }
      const bool zero = l == 0.0f;  // nothing seen: O is 0 whatever the accumulator holds
      const int slot = cta * 2 + (s.k0 > 0 ? 0 : 1);  // a piece that starts inside its unit is the first
      const int prow = (pair ? t * 128 : 0) + r;      // row of the piece
      const int prows = pair ? 256 : 128;
      float4* part = reinterpret_cast<float4*>(p.o_part + static_cast<int64_t>(slot) * prows * D) + prow;
      // Rows of this lane's quad in O, from the tile's first query (-1: no row).
      T* out = reinterpret_cast<T*>(p.o) + ((static_cast<int64_t>(s.b) * p.T + (qi - div_g(r))) * p.Hq + s.hk * p.g) * D;
      int orow[4], rrq = div_g(r & ~3), rhg = (r & ~3) - rrq * p.g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        orow[i] = rrq < p.qpt && qi - div_g(r) + rrq < p.T ? (rrq * p.Hq + rhg) * D : -1;
        if (++rhg == p.g) rhg = 0, ++rrq;
      }
      const bool mine = t < live;  // two tiles: this warpgroup's tile is in use
      if (n > 0 && (!pair || mine)) {
        const int tt = pair ? t : 0;
        ok = __all_sync(0xffffffffu, w.wait(&sm.o_final[tt], (oph >> tt) & 1, kErrTreeWait)) &&
             (pair || n == 1 || __all_sync(0xffffffffu, w.wait(&sm.o_final[1], oph >> 1, kErrTreeWait)));
        if (!ok) break;
      }
      if (n > 0) oph ^= live == 2 ? 3u : 1u;
      tc_fence_after();
      // 32 columns from column c on, in registers, to O or to the piece.
      auto put = [&](int c, const float* v) {
        if (s.whole) {
          // A thread's 32 columns of its own row would go out 16 bytes to 32
          // far apart rows at a time: the four lanes of a quad exchange their
          // 16-byte pieces (a 4 x 4 transpose) and each store of the warp
          // covers 64 bytes of 8 rows.
          uint32_t w16[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w16[e] = BF16 ? pack_bf16(v[2 * e], v[2 * e + 1]) : pack_f16(v[2 * e], v[2 * e + 1]);
          quad_transpose(w16, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)  // row (r & ~3) + i, piece lane & 3
            if (orow[i] >= 0)
              *reinterpret_cast<uint4*>(out + orow[i] + c + 8 * (lane & 3)) =
                  make_uint4(w16[4 * i], w16[4 * i + 1], w16[4 * i + 2], w16[4 * i + 3]);
          __syncwarp();
        } else if (row_in) {
          // [D / 4][rows][4]: a warp's 32 rows are one 512-byte line.
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            part[(c + i) / 4 * prows] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      };
      // O is read whole, in one wait, and handed back before it is packed.
      if (n == 0) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
#pragma unroll 1
        for (int c = pair ? 0 : t * (D / 2); c < (pair ? D : (t + 1) * (D / 2)); c += 32) put(c, v);
      } else if (pair) {
        // 32 columns at a time: with all of O in registers the row pointers spill
        // (16 sequences, 64 nodes, 4096 keys: 78.5 against 80.3 us).
        if (mine) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t ov[32];
            tmem_ld32(tmem + C::tm_o(t) + lane_base + c, ov);
            tmem_ld_wait();
            reg_fence(ov);
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = zero ? 0.0f : __uint_as_float(ov[i]) * scale0;
            put(c, v);
          }
        }
        tc_fence_before();
        mbar_arrive(&sm.o_free[t]);
        ++seg;
      } else {
        // Half the columns of both streams' accumulators.
        const bool one = n == 1;  // the second stream had no tile
#pragma unroll 1
        for (int c = t * (D / 2); c < (t + 1) * (D / 2); c += 32) {
          uint32_t o0[32], o1[32];
          tmem_ld32(tmem + C::tm_o(0) + lane_base + c, o0);
          tmem_ld32(tmem + C::tm_o(1) + lane_base + c, o1);
          tmem_ld_wait();
          reg_fence(o0);
          reg_fence(o1);
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float x = __uint_as_float(o0[i]) * scale0;
            v[i] = zero ? 0.0f : one ? x : fmaf(__uint_as_float(o1[i]), scale1, x);
          }
          put(c, v);
        }
        tc_fence_before();
        mbar_arrive(&sm.o_free[0]);
        mbar_arrive(&sm.o_free[1]);
        ++seg;
      }
      if (row_in && (pair ? mine || n == 0 : t == 0)) {
        if (s.whole) {
          if (p.lse != nullptr) p.lse[(static_cast<int64_t>(s.b) * p.Hq + hq) * p.T + qi] = lse;
        } else {
          p.ml_part[static_cast<int64_t>(slot) * prows + prow] = make_float2(zero ? -INFINITY : m, l);
        }
      }
      tree_release(sm, dk);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// Merges the pieces of every unit that was cut: block x does it where CTA x of the
// tree kernel is the first to begin inside a unit (p.cut), blockIdx.y picks 8
// columns, a thread is a row.
//   M = max m_i, O = sum 2^(m_i - M) O_i / (sum 2^(m_i - M) l_i [+ 2^(sink - M)])
// A unit has up to as many pieces as there are CTAs (one sequence with one kv head;
// some twenty with eight), which one thread reads one after the other: latency
// bound, hence narrow column slices, four pieces in flight and one pass with a
// running maximum.  (One user with 131072 keys, d = 128, both kernels: 46 us with
// one kv head, 52 with two, 112 with eight; reading K and V takes 10, 20 and 79.)
// It is launched with programmatic serialisation, so that only its first read
// waits for the tree kernel.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_tree_merge_kernel(const __grid_constant__ TreeParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  pdl_wait();
  const int4 cut = p.cut[blockIdx.x];
  if (cut.x < 0) return;
  const int b = cut.x, rb = cut.y / p.Hkv, hk = cut.y - rb * p.Hkv;
  const int prows = p.two_tiles ? 256 : 128;
  const int row = threadIdx.x;  // blockDim.x == prows
  const int t = row >> 7, r = row & 127;
  const int rq = r / p.g, hg = r - rq * p.g;
  const int qi = rb * (p.two_tiles ? 2 : 1) * p.qpt + t * p.qpt + rq;
  if (rq >= p.qpt || qi >= p.T) return;
  const int hq = hk * p.g + hg;
  const int c0 = blockIdx.x - 1, n = cut.z - c0 + 1, col = blockIdx.y * 8;
  auto piece = [&](int i) { return static_cast<int64_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)); };
  float M = p.sink != nullptr ? p.sink[hq] * kLog2e : -INFINITY;
  float z = p.sink != nullptr ? 1.0f : 0.0f;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 4) {
    float2 e[4];
    float4 v0[4], v1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = make_float2(-INFINITY, 0.0f);
      v0[i] = v1[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i0 + i < n) {
        const int64_t q = piece(i0 + i);
        const float4* part = reinterpret_cast<const float4*>(p.o_part + q * prows * D) + (col / 4) * prows + row;
        e[i] = p.ml_part[q * prows + row];
        v0[i] = part[0];
        v1[i] = part[prows];
      }
    }
    const float m = fmaxf(fmaxf(M, fmaxf(e[0].x, e[1].x)), fmaxf(e[2].x, e[3].x));
    const float ms = m == -INFINITY ? 0.0f : m;
    const float a = ex2_approx(M - ms);
    M = m;
    z *= a;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= a;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float wgt = ex2_approx(e[i].x - ms);
      z = fmaf(e[i].y, wgt, z);
      acc[0] = fmaf(v0[i].x, wgt, acc[0]);
      acc[1] = fmaf(v0[i].y, wgt, acc[1]);
      acc[2] = fmaf(v0[i].z, wgt, acc[2]);
      acc[3] = fmaf(v0[i].w, wgt, acc[3]);
      acc[4] = fmaf(v1[i].x, wgt, acc[4]);
      acc[5] = fmaf(v1[i].y, wgt, acc[5]);
      acc[6] = fmaf(v1[i].z, wgt, acc[6]);
      acc[7] = fmaf(v1[i].w, wgt, acc[7]);
    }
  }
  const float norm = z != 0.0f ? 1.0f / z : 0.0f;  // (a NaN piece makes z NaN, and so the row)
  T* out = reinterpret_cast<T*>(p.o) + ((static_cast<int64_t>(b) * p.T + qi) * p.Hq + hq) * D + col;
  uint32_t w4[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float lo = acc[2 * e] * norm, hi = acc[2 * e + 1] * norm;
    w4[e] = BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
  }
  *reinterpret_cast<uint4*>(out) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
  if (col == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.T + qi] = z != 0.0f ? (M + __log2f(z)) * kLn2 : -INFINITY;
}

template <int D, bool BF16, bool SOFTCAP, bool pair>
static cudaError_t launch_tree_t(const TreeParams& p, cudaStream_t stream) {
  using C = TreeCfg<D>;
  auto kern = attn_tree_kernel<D, BF16, SOFTCAP, pair>;
  const int smem = static_cast<int>(sizeof(TreeSmem<C>));
  static_assert(sizeof(TreeSmem<C>) <= 227 * 1024, "shared memory per block");
  // setmaxnreg.inc draws on what the block was launched with: refuse to launch
  // a build whose launch count is not the one the split assumes.
  static std::atomic<uint64_t> configured{0};  // bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_relaxed) & bit)) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != C::LAUNCH_REGS) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  e = launch_pdl(kern, dim3(p.grid), C::THREADS, smem, stream, p);
  if (e != cudaSuccess || p.o_part == nullptr) return e;
  return launch_pdl(attn_tree_merge_kernel<D, BF16>, dim3(p.grid, D / 8), p.two_tiles ? 256 : 128, 0, stream, p);
}

template <bool BF16, bool SOFTCAP>
static cudaError_t launch_tree_p(const TreeParams& p, cudaStream_t stream) {
  return p.two_tiles ? launch_tree_t<ATTN_TREE_D, BF16, SOFTCAP, true>(p, stream)
                     : launch_tree_t<ATTN_TREE_D, BF16, SOFTCAP, false>(p, stream);
}

template <>
cudaError_t launch_tree_d<ATTN_TREE_D>(const TreeParams& p, bool bf16, bool softcap, cudaStream_t stream) {
  if (bf16) return softcap ? launch_tree_p<true, true>(p, stream) : launch_tree_p<true, false>(p, stream);
  return softcap ? launch_tree_p<false, true>(p, stream) : launch_tree_p<false, false>(p, stream);
}

}  // namespace attn
