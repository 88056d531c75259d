// linear_kernel.cuh -- linear attention with a decay per head, in chunks of 128
// tokens on the tensor cores.
//
// With w = e^g and S the state before a chunk of C tokens (rows 0 .. C - 1 of it):
//   o_i = scale * ( sum_{j <= i} w^(i-j) (q_i . k_j) v_j  +  w^(i+1) q_i^T S )
//   S  <- w^C S + sum_j w^(C-1-j) k_j v_j^T
// that is four products per chunk: Q K^T, the weights P times V, Q S, and K^T V'
// with V' = w^(C-1-j) v_j.  A CTA walks the chunks of one head for 64 columns of
// v (the columns of S are independent); the CTAs of a head's two halves run next
// to each other and share Q and K in L2.
//
// What bounds it: a chunk moves 80 KB (d = 128) for 12.6 MFLOP, 1536 cycles of the
// tensor core against some 1900 of its share of HBM, so everything else has to hide
// behind those: three groups of four warps and two warps to issue loads and products.
//   weights  (thread = row): Q K^T from tensor memory, decays, mask, P back into tensor
//            memory, over the columns it came from.
//   state    (thread = row of S): S from tensor memory, rounded into shared memory as
//            the operand of Q S, and back times w^C before K^T V' adds to it.
//   values   (thread = token): V' into shared memory in two pieces; rows behind the
//            sequence's end cleared.
//   output   (the same warps, thread = row): both parts of o from tensor memory, stored.
//
// Roundings to 16 bits: P and the operand copy of S, each at most half a step of
// the type, as o itself is.  The state proper stays in 32 bits in tensor memory, and what is added
// to it is V' in two pieces (v' = hi + lo, lo's own rounding 2^-18 of v' in bf16): one piece would
// put a 16-bit error into a 32-bit result that later calls build on.  fp16 has no room for either
// operand's range: the rows of P and the copy of S are scaled by powers of two to fit.
//
// Few sequences and heads leave SMs idle.  Then the chunks are cut into segments
// (linear_segments in linear.h): a first launch (STATES) adds up the state every segment
// but the last contributes, with decays taken to the segment's end so that nothing is rescaled on the way, and the
// second starts each segment from the decayed sum of those before it.
#pragma once
#include "ptx.cuh"
#include "linear.h"
#include "launch.h"
#include "softmax.cuh"

namespace attn {

template <int D>
struct LinearCfg {
  static constexpr int C = kLinearChunk;
  static constexpr int N = 64;                    // columns of v per CTA
  static constexpr int NCHUNK = D / 64;           // swizzle atoms along d
  static constexpr int TILE = C * D * 2;          // a Q or K tile
  static constexpr int ATOM = C * 128;            // one 64-column atom of it, and a V tile
  static constexpr int THREADS = 14 * 32;
  static constexpr int W_TMA = 12, W_MMA = 13;
  // Tensor memory: chunk n's S = Q K^T at 128 (n & 1) with P over its first and
  // P V over its last 64 columns, Q S at 256 + 64 (n & 1), the state at 384.
  static constexpr uint32_t TM_COLS = 512;
  __device__ static constexpr uint32_t tm_s(int b) { return 128u * b; }
  __device__ static constexpr uint32_t tm_pv(int b) { return 128u * b + 64u; }
  __device__ static constexpr uint32_t tm_qs(int b) { return 256u + 64u * b; }
  static constexpr uint32_t TM_STATE = 384;
};

template <int D>
struct LinearSmem {
  using C = LinearCfg<D>;
  alignas(1024) uint8_t q[2][C::TILE];
  alignas(1024) uint8_t k[2][C::TILE];
  alignas(1024) uint8_t v[2][C::ATOM];
  alignas(1024) uint8_t vp[2][C::ATOM];  // V', first and second piece
  alignas(1024) uint8_t sb[D * 128];     // the state as an operand
  alignas(1024) uint4 ostage[4][32 * 8];
  float row_scale[2][128];  // fp16: what the rows of P were divided by
  float state_scale[4];     // and the state (read up to two chunks late)
  float pw[64];             // [31 + n]: w^n for n >= 0, else 0
  float col[32];            // [j]: w^(31 - j)
  uint64_t qk_full[2], qk_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t sb_full, sb_empty, kv_done, vp_full, teardown;
  uint32_t tmem_base;
  uint32_t part[4];
  int abort_flag;
};

__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// w^n for n >= 0 from log2 w (w = 0: 1, 0, 0, ...).
__device__ __forceinline__ float decay_pow(float log2w, int n) { return n == 0 ? 1.0f : exp2f(log2w * n); }

// 2^e and 2^-e such that m 2^-e is at most 2^top (m = 0, infinity or NaN: 1).
__device__ __forceinline__ void fit(float m, int top, float& up, float& down) {
  const int e0 = static_cast<int>(__float_as_uint(m) >> 23);  // (m >= 0)
  int e = e0 == 0 || e0 >= 255 ? 0 : e0 - 126 - top;
  e = max(-100, min(e, 120));
  up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}
template <bool BF16>
__device__ __forceinline__ void unpack16(uint32_t w, float& lo, float& hi) {
  if constexpr (BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    lo = __low2float(h);
    hi = __high2float(h);
  }
}

template <int D, bool BF16, bool STATES>
__global__ void __launch_bounds__(LinearCfg<D>::THREADS, 1) linear_chunk_kernel(const __grid_constant__ LinearParams p) {
  using C = LinearCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  LinearSmem<D>& sm =
      *reinterpret_cast<LinearSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = blockIdx.x, h = blockIdx.y, b = blockIdx.z / p.segs, seg = blockIdx.z - b * p.segs;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.qk_full[i], 1);
      mbar_init(&sm.qk_empty[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.o_empty[i], 128);
    }
    mbar_init(&sm.sb_full, 128);
    mbar_init(&sm.sb_empty, 1);
    mbar_init(&sm.kv_done, 1);
    mbar_init(&sm.vp_full, 128);
    mbar_init(&sm.teardown, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  const int slot = state_of(p.index, p.num_states, b, p.err, half == 0 && h == 0 && seg == 0);
  int row0, len;
  sequence_rows(p, b, row0, len);
  // This CTA's tokens: [t0, t1) of the sequence.
  const int seg_len = p.seg_chunks * C::C;  // (chunks of all segments fit an int: see the launch)
  const int t0 = seg * seg_len;
  const int t1 = seg == p.segs - 1 ? len : min(len, t0 + seg_len);
  const bool last = t1 >= len;  // of its sequence
  // A later segment without tokens has nothing to do; the first launch leaves the
  // last one of each sequence out.
  if ((t0 >= len && seg > 0) || (STATES && last)) return;
  const int chunks = (t1 - t0 + C::C - 1) / C::C;
  const float log2w = p.log_decay[h] * kLog2e;
  if (tid < 64) sm.pw[tid] = tid < 31 ? 0.0f : decay_pow(log2w, tid - 31);
  else if (tid < 96) sm.col[tid - 64] = decay_pow(log2w, 95 - tid);
  if (warp == C::W_MMA) {
    tmem_alloc(&sm.tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const Waiter w{globaltimer_ns() + p.timeout_ns, &sm.abort_flag, p.err};
  const int hk = h / p.group, bc = p.cu != nullptr ? 0 : b;
  const int64_t head = static_cast<int64_t>(D) * D;
  const int64_t work_seg = static_cast<int64_t>(p.B) * p.Hq * head;  // floats of a segment's states
  const int64_t work_at = (static_cast<int64_t>(b) * p.Hq + h) * head + half * C::N;

  if (warp == C::W_TMA) {
    // ===================== loads ==============================================
    if (lane == 0) {
      int qk_armed = 0, v_armed = 0;
      bool ok = true;
      auto row_of = [&](int n) { return row0 + t0 + n * C::C; };
      for (int n = 0; n < chunks; ++n) {
        const int s = n & 1;
        const uint32_t ph = ((n >> 1) & 1) ^ 1;
        if (!(ok = w.wait(&sm.qk_empty[s], ph, kErrLinearWait))) break;
        mbar_arrive_expect_tx(&sm.qk_full[s], STATES ? C::TILE : 2 * C::TILE);
        ++qk_armed;
#pragma unroll
        for (int c = 0; c < C::NCHUNK; ++c) {
          tma_load_4d(sm.k[s] + c * C::ATOM, &p.tm_k, &sm.qk_full[s], c * 64, row_of(n), hk, bc);
          if constexpr (!STATES) tma_load_4d(sm.q[s] + c * C::ATOM, &p.tm_q, &sm.qk_full[s], c * 64, row_of(n), h, bc);
        }
        if (!(ok = w.wait(&sm.v_empty[s], ph, kErrLinearWait))) break;
        mbar_arrive_expect_tx(&sm.v_full[s], C::ATOM);
        ++v_armed;
        tma_load_4d(sm.v[s], &p.tm_v, &sm.v_full[s], half * C::N, row_of(n), hk, bc);
      }
      if (w.aborted()) {  // every copy started must land before shared memory is released
        const uint64_t dl = globaltimer_ns() + 50000000ull;
        for (int i = max(0, qk_armed - 2); i < qk_armed; ++i) wait_raw(&sm.qk_full[i & 1], (i >> 1) & 1, dl);
        for (int i = max(0, v_armed - 2); i < v_armed; ++i) wait_raw(&sm.v_full[i & 1], (i >> 1) & 1, dl);
      }
    }
  } else if (warp == C::W_MMA) {
    // ===================== products (whole warp, one lane issues) ==============
    const uint32_t lead = elect_one() ? 1u : 0u;
    constexpr uint32_t id_s = idesc_f16_f32(BF16, 128, 128, false, false);
    constexpr uint32_t id_pv = idesc_f16_f32(BF16, 128, 64, false, true);
    constexpr uint32_t id_kv = idesc_f16_f32(BF16, 128, 64, true, true);
    const uint64_t qd0 = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024), kd0 = sdesc_sw128(smem_u32(sm.k[0]), 16, 1024);
    // d = 64: the second 64 rows of K^T re-read the first (leading offset 0), and rows
    // 64 .. 127 of S are ignored.
    const uint64_t ktd0 = sdesc_sw128(smem_u32(sm.k[0]), C::NCHUNK > 1 ? C::ATOM : 0, 1024);
    const uint64_t vd0 = sdesc_sw128(smem_u32(sm.v[0]), C::ATOM, 1024);
    const uint64_t vpd0 = sdesc_sw128(smem_u32(sm.vp[0]), C::ATOM, 1024);
    const uint64_t sbd = sdesc_sw128(smem_u32(sm.sb), C::ATOM, 1024);
    auto issue_s = [&](int n) {
      const uint64_t st = static_cast<uint64_t>((n & 1) * (C::TILE >> 4));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t off = ((i >> 2) * C::ATOM + (i & 3) * 32) >> 4;
        umma_ss_warp(tmem + C::tm_s(n & 1), qd0 + st + off, kd0 + st + off, id_s, i > 0 ? 1u : 0u, lead);
      }
      umma_commit_warp(&sm.s_full[n & 1], lead);
    };
    bool ok = true;
    if (chunks > 0) {
      ok = w.wait(&sm.qk_full[0], 0, kErrLinearWait);
      tc_fence_after();
      if (!STATES && ok) issue_s(0);
    }
    for (int n = 0; ok && n < chunks; ++n) {
      const int s = n & 1;
      // S += K^T V'
      if (!(ok = w.wait(&sm.vp_full, n & 1, kErrLinearWait))) break;
      if (STATES ? n == 0 : true)
        if (!(ok = w.wait(&sm.sb_full, STATES ? 0 : n & 1, kErrLinearWait))) break;
      if (STATES && !(ok = w.wait(&sm.qk_full[s], (n >> 1) & 1, kErrLinearWait))) break;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < C::C / 16; ++i) {
        const uint64_t ka = ktd0 + static_cast<uint64_t>(s * (C::TILE >> 4) + ((i * 16 * 128) >> 4));
        umma_ss_warp(tmem + C::TM_STATE, ka, vpd0 + ((i * 16 * 128) >> 4), id_kv, 1u, lead);
        umma_ss_warp(tmem + C::TM_STATE, ka, vpd0 + ((C::ATOM + i * 16 * 128) >> 4), id_kv, 1u, lead);
      }
      umma_commit_warp(&sm.kv_done, lead);
      if constexpr (STATES) {
        umma_commit_warp(&sm.qk_empty[s], lead);
        umma_commit_warp(&sm.v_empty[s], lead);
      } else {
        // Q S (its columns are free: S of this chunk waited for them)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          umma_ss_warp(tmem + C::tm_qs(s), qd0 + static_cast<uint64_t>(s * (C::TILE >> 4) + (((i >> 2) * C::ATOM + (i & 3) * 32) >> 4)),
                       sbd + ((i * 16 * 128) >> 4), id_pv, i > 0 ? 1u : 0u, lead);
        umma_commit_warp(&sm.sb_empty, lead);
        umma_commit_warp(&sm.qk_empty[s], lead);
        if (n + 1 < chunks) {
          if (!(ok = w.wait(&sm.qk_full[s ^ 1], ((n + 1) >> 1) & 1, kErrLinearWait))) break;
          if (n >= 1 && !(ok = w.wait(&sm.o_empty[s ^ 1], ((n - 1) >> 1) & 1, kErrLinearWait))) break;
          tc_fence_after();
          issue_s(n + 1);
        }
        // P V
        if (!(ok = w.wait(&sm.p_full[s], (n >> 1) & 1, kErrLinearWait))) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < C::C / 16; ++i)
          umma_ts_warp(tmem + C::tm_pv(s), tmem + C::tm_s(s) + i * 8,
                       vd0 + static_cast<uint64_t>(s * (C::ATOM >> 4) + ((i * 16 * 128) >> 4)), id_pv, i > 0 ? 1u : 0u, lead);
        umma_commit_warp(&sm.o_full[s], lead);
        umma_commit_warp(&sm.v_empty[s], lead);
      }
    }
    if constexpr (STATES) umma_commit_warp(&sm.o_full[0], lead);  // the segment's state is complete
    // All products must be done before tensor memory is freed.
    umma_commit_warp(&sm.teardown, lead);
    if (!wait_raw(&sm.teardown, 0, globaltimer_ns() + 50000000ull) && p.err) atomicOr(p.err, 1u << kErrLinearTeardown);
  } else if (warp < 4) {
    // ===================== weights: P_ij = scale w^(i-j) q_i . k_j ==============
    if constexpr (!STATES) {
      const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
      bool ok = true;
      for (int n = 0; ok && n < chunks; ++n) {
        ok = __all_sync(0xffffffffu, w.wait(&sm.s_full[n & 1], (n >> 1) & 1, kErrLinearWait));
        if (!ok) break;
        tc_fence_after();
        const uint32_t base = tmem + C::tm_s(n & 1) + lanes;
        float f = p.scale;
        if constexpr (!BF16) {
          // fp16: the row's largest score decides a power of two that fits its weights (at
          // most 2^11: room for decays a little above 1, and 2^35 below for the small).
          float m = 0.0f;
#pragma unroll 1
          for (int cb = 0; cb <= warp; ++cb) {
            uint32_t r[32];
            tmem_ld32(base + 32 * cb, r);
            tmem_ld_wait();
            reg_fence(r);
            const int seen = cb < warp ? 31 : lane;
#pragma unroll
            for (int j = 0; j < 32; ++j) m = fmaxf(m, j <= seen ? fabsf(__uint_as_float(r[j])) : 0.0f);
          }
          float up, down;
          fit(m * p.scale, 11, up, down);
          sm.row_scale[n & 1][tid] = up;
          f *= down;
        }
        uint32_t pk[16];
        // Blocks of 32 columns left of the diagonal one: w^(i-j) is the row's power down to
        // the block's last column times the column's from there.  (From the left: a block's
        // weights go where the one before it was read.)
#pragma unroll 1
        for (int cb = 0; cb < warp; ++cb) {
          uint32_t r[32];
          tmem_ld32(base + 32 * cb, r);
          tmem_ld_wait();
          reg_fence(r);
          const float rowf = f * exp2f(log2w * (lane + 1 + 32 * (warp - 1 - cb)));
          const uint64_t f2 = f2_pack(rowf, rowf);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 c = *reinterpret_cast<const float4*>(&sm.col[j]);
            float x0, x1, x2, x3;
            f2_unpack(f2_mul(f2_mul(f2_pack(c.x, c.y), f2), f2_pack(__uint_as_float(r[j]), __uint_as_float(r[j + 1]))),
                      x0, x1);
            f2_unpack(f2_mul(f2_mul(f2_pack(c.z, c.w), f2), f2_pack(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]))),
                      x2, x3);
            pk[j / 2] = pack16<BF16>(x0, x1);
            pk[j / 2 + 1] = pack16<BF16>(x2, x3);
          }
          tmem_st16(base + 16 * cb, pk);
        }
        {
          uint32_t r[32];
          tmem_ld32(base + 32 * warp, r);
          tmem_ld_wait();
          reg_fence(r);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float a = __uint_as_float(r[j]) * (f * sm.pw[31 + lane - j]);
            const float c = __uint_as_float(r[j + 1]) * (f * sm.pw[30 + lane - j]);
            pk[j / 2] = pack16<BF16>(j <= lane ? a : 0.0f, j + 1 <= lane ? c : 0.0f);
          }
          tmem_st16(base + 16 * warp, pk);
        }
        if (warp < 3) {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = 0u;
#pragma unroll 1
          for (int cb = warp + 1; cb < 4; ++cb) tmem_st16(base + 16 * cb, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.p_full[n & 1]);
      }
    }
  } else if (warp < 8) {
    // ===================== state: thread = row of S =============================
    const int r = tid - 128, wq = warp - 4;
    const uint32_t at = tmem + C::TM_STATE + (static_cast<uint32_t>(wq * 32) << 16);
    const bool mine = D == 128 || wq < 2;  // (d = 64: rows 64 .. 127 of tensor memory hold nothing)
    float s[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) s[i] = 0.0f;
    auto add = [&](const float* from, float f) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(from + 4 * i);
        s[4 * i] = fmaf(x.x, f, s[4 * i]);
        s[4 * i + 1] = fmaf(x.y, f, s[4 * i + 1]);
        s[4 * i + 2] = fmaf(x.z, f, s[4 * i + 2]);
        s[4 * i + 3] = fmaf(x.w, f, s[4 * i + 3]);
      }
    };
    auto put = [&](float* to) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float4*>(to + 4 * i) = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    };
    const int64_t state_at = (static_cast<int64_t>(slot) * p.Hq + h) * head + half * C::N + r * D;
    const bool has_in = p.state_in != nullptr && slot >= 0;
    if (mine) {
      if (seg == 0 && has_in) {
        // (Cut sequences: state_out may be state_in, whose last segment may be done before
        // this one starts: it is read from where the first launch has put it.)
        add(STATES || last ? p.state_in + state_at : p.work + (p.segs - 1) * work_seg + work_at + r * D, 1.0f);
        if constexpr (STATES) put(p.work + (p.segs - 1) * work_seg + work_at + r * D);
      } else if (!STATES && seg > 0) {
        for (int i = seg - 1; i >= 0; --i) {
          const float f = decay_pow(log2w, (seg - 1 - i) * seg_len);
          if (f == 0.0f) break;
          add(p.work + i * work_seg + work_at + r * D, f);
        }
      }
    }
    bool ok = true;
    // Waits until the products so far are in S.
    auto reach = [&](uint64_t* bar, int phase) {
      ok = __all_sync(0xffffffffu, w.wait(bar, phase & 1, kErrLinearWait));
      tc_fence_after();
    };
    auto start = [&](float f) {  // S times f into tensor memory
      if (!mine) return;
#pragma unroll
      for (int i = 0; i < 64; i += 32) {
        uint32_t a[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] = __float_as_uint(s[i + j] * f);
        tmem_st32(at + i, a);
      }
      tmem_st_wait();
    };
    auto finish = [&](float* to) {
      if (!mine) return;
#pragma unroll 1
      for (int i = 0; i < 64; i += 32) {
        uint32_t a[32];
        tmem_ld32(at + i, a);
        tmem_ld_wait();
        reg_fence(a);
#pragma unroll
        for (int j = 0; j < 32; j += 4) *reinterpret_cast<uint4*>(to + i + j) = make_uint4(a[j], a[j + 1], a[j + 2], a[j + 3]);
      }
    };
    if constexpr (STATES) {
      start(decay_pow(log2w, t1 - t0));
      tc_fence_before();
      mbar_arrive(&sm.sb_full);
      reach(&sm.o_full[0], 0);
      if (ok) finish(p.work + seg * work_seg + work_at + r * D);
    } else {
      start(1.0f);
      const float full = decay_pow(log2w, C::C);
      uint8_t* row = sm.sb + r * 128;
      for (int n = 0; ok && n < chunks; ++n) {
        if (n > 0) reach(&sm.kv_done, n - 1);
        float down = 1.0f;
        if constexpr (!BF16) {
          // fp16: one power of two for the whole operand, its largest element below 2^15.
          float m = 0.0f;
          if (mine) {
#pragma unroll 1
            for (int i = 0; i < 64; i += 32) {
              uint32_t a[32];
              tmem_ld32(at + i, a);
              tmem_ld_wait();
              reg_fence(a);
#pragma unroll
              for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(__uint_as_float(a[j])));
            }
          }
          const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
          if (lane == 0) sm.part[wq] = top;
          // (Every thread comes here, aborted or not, and all leave together.)
          ok = !named_bar_or(1, 128, !ok);
          m = __uint_as_float(max(max(sm.part[0], sm.part[1]), max(sm.part[2], sm.part[3])));
          float up;
          fit(m, 15, up, down);
          if (r == 0) sm.state_scale[n & 3] = up;
        }
        if (ok && n > 0) ok = __all_sync(0xffffffffu, w.wait(&sm.sb_empty, (n - 1) & 1, kErrLinearWait));
        if constexpr (!BF16) ok = !named_bar_or(1, 128, !ok);  // (also: sm.part has been read)
        if (!ok) break;
        const int m = t1 - t0 - n * C::C;
        const float f = m >= C::C ? full : decay_pow(log2w, m);
        if (mine) {
#pragma unroll 1
          for (int i = 0; i < 64; i += 32) {
            uint32_t a[32];
            tmem_ld32(at + i, a);
            tmem_ld_wait();
            reg_fence(a);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float lo = __uint_as_float(a[8 * j + 2 * e]), hi = __uint_as_float(a[8 * j + 2 * e + 1]);
                if constexpr (!BF16) lo *= down, hi *= down;
                x[e] = pack16<BF16>(lo, hi);
              }
              *reinterpret_cast<uint4*>(row + (((i / 8 + j) ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) * f);
            tmem_st32(at + i, a);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        fence_proxy_async_smem();
        mbar_arrive(&sm.sb_full);
      }
      if (ok && last && chunks > 0) reach(&sm.kv_done, chunks - 1);
      if (ok && last && p.state_out != nullptr && slot >= 0) finish(p.state_out + state_at);
    }
  } else if (warp < 12) {
    // ===================== values and output =====================================
    // Chunk n's V' (thread = token), then chunk n - 1's o (thread = row): the products
    // that need V' come first, and o's of the chunk before end about then.
    const int r = tid - 256, wq = warp - 8;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const float since = p.scale * decay_pow(log2w, r + 1);
    const float ahead = decay_pow(log2w, C::C - 1 - r);
    uint16_t* out = static_cast<uint16_t*>(p.o) + bc * p.o_batch + h * p.o_head + half * C::N;
    uint4* stage = sm.ostage[wq];
    bool ok = true;
    // V' = w^(tokens behind it up to where the state is wanted) v: to the chunk's end,
    // in the first launch to the segment's.
    auto values = [&](int n) {
      const int st = n & 1;
      ok = __all_sync(0xffffffffu, w.wait(&sm.v_full[st], (n >> 1) & 1, kErrLinearWait));
      if (ok && n > 0) ok = __all_sync(0xffffffffu, w.wait(&sm.kv_done, (n - 1) & 1, kErrLinearWait));
      if (!ok) return;
      const int left = t1 - t0 - n * C::C;  // tokens from this chunk on
      const int live = min(left, C::C);
      const float f = !STATES && live == C::C ? ahead
                      : r < live              ? decay_pow(log2w, (STATES ? left : live) - 1 - r)
                                              : 0.0f;
      uint8_t* src = sm.v[st] + r * 128;
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        const int at = (i ^ (r & 7)) << 4;
        const uint4 x = *reinterpret_cast<const uint4*>(src + at);
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a, c, ah, ch;
          unpack16<BF16>(r < live ? in[e] : 0u, a, c);  // (rows of nobody may hold anything)
          a *= f;
          c *= f;
          hi[e] = pack16<BF16>(a, c);
          unpack16<BF16>(hi[e], ah, ch);
          lo[e] = pack16<BF16>(a - ah, c - ch);
        }
        *reinterpret_cast<uint4*>(sm.vp[0] + r * 128 + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(sm.vp[1] + r * 128 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      if (live < C::C) {
        // What lies behind the end meets weights of 0, and 0 * NaN is not 0.
        ok = __all_sync(0xffffffffu, w.wait(&sm.qk_full[st], (n >> 1) & 1, kErrLinearWait));
        if (!ok) return;
        if (r >= live) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            *reinterpret_cast<uint4*>(src + i * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < C::NCHUNK; ++c)
              *reinterpret_cast<uint4*>(sm.k[st] + c * C::ATOM + r * 128 + i * 16) = make_uint4(0, 0, 0, 0);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sm.vp_full);
    };
    auto output = [&](int n) {
      ok = __all_sync(0xffffffffu, w.wait(&sm.o_full[n & 1], (n >> 1) & 1, kErrLinearWait));
      if (!ok) return;
      tc_fence_after();
      float fi = 1.0f, fs = since;
      if constexpr (!BF16) {
        fi = sm.row_scale[n & 1][r];
        fs *= sm.state_scale[n & 3];
      }
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        uint32_t a[32], x[32];
        tmem_ld32(tmem + C::tm_pv(n & 1) + lanes + c, a);
        tmem_ld32(tmem + C::tm_qs(n & 1) + lanes + c, x);
        tmem_ld_wait();
        reg_fence(a);
        reg_fence(x);
        const uint64_t fs2 = f2_pack(fs, fs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 8 * i + 2 * e;
            uint64_t o2 = f2_pack(__uint_as_float(a[j]), __uint_as_float(a[j + 1]));
            if constexpr (!BF16) o2 = f2_mul(o2, f2_pack(fi, fi));
            o2 = f2_fma(f2_pack(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), fs2, o2);
            float lo, hi;
            f2_unpack(o2, lo, hi);
            pk[e] = pack16<BF16>(lo, hi);
          }
          stage[lane * 8 + ((c / 8 + i) ^ (lane & 7))] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
      tc_fence_before();
      mbar_arrive(&sm.o_empty[n & 1]);
      __syncwarp();
      const int first = t0 + n * C::C;
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {
        const int rw = 4 * i + (lane >> 3), q = lane & 7, t = first + wq * 32 + rw;
        if (t < t1)
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row0 + t) * p.o_row + q * 8) =
              stage[rw * 8 + (q ^ (rw & 7))];
      }
      __syncwarp();
    };
    for (int n = 0; ok && n < chunks; ++n) {
      values(n);
      if constexpr (!STATES)
        if (ok && n > 0) output(n - 1);
    }
    if constexpr (!STATES)
      if (ok && chunks > 0) output(chunks - 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

template <int D, bool BF16, bool STATES>
static cudaError_t launch_linear_t(const LinearParams& p, int segs, cudaStream_t stream) {
  constexpr size_t smem = sizeof(LinearSmem<D>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory per block");
  const dim3 grid(D / 64, static_cast<unsigned>(p.Hq), static_cast<unsigned>(p.B) * segs);
  return launch_pdl_upto<linear_chunk_kernel<D, BF16, STATES>>(smem, grid, LinearCfg<D>::THREADS, smem, stream, p);
}

template <int D, bool BF16>
static cudaError_t launch_linear_b(const LinearParams& p, cudaStream_t stream) {
  if (p.segs > 1) {
    const cudaError_t e = launch_linear_t<D, BF16, true>(p, p.segs, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_linear_t<D, BF16, false>(p, p.segs, stream);
}

template <>
cudaError_t launch_linear_d<ATTN_LINEAR_D>(const LinearParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_linear_b<ATTN_LINEAR_D, true>(p, stream) : launch_linear_b<ATTN_LINEAR_D, false>(p, stream);
}

}  // namespace attn
