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
// Measured: 2 x 8192 tokens of 32 heads, d = 128, bf16 in 101 us, 5.3 TB/s (0.80 of a copy's
// rate; fp16 130, its operands scaled into range); 16 heads of 2048 in 22.7 (fp16 25.8).
//
// What bounds it: a chunk moves 80 KB (d = 128) for 12.6 MFLOP, 1536 cycles of the
// tensor core against some 1900 of its share of HBM, so everything else has to hide
// behind those.  The chain from chunk to chunk is K^T V' -> S from tensor memory, as operand and
// back times w^C -> K^T V'; all other work is kept off it by warps of their own:
//   state, output   (8 warps, thread = row and 32 columns): S rounded into shared memory as
//            the operand of Q S, and back times w^C before K^T V' adds to it; then both
//            parts of the o of the chunk before, stored.
//   values, weights (8 warps): V' in two pieces (thread = token), worked out in registers while
//            the products still read the one before; rows behind the sequence's end cleared.
//            Then Q K^T from tensor memory (thread = row), decays, mask, P back into
//            tensor memory over the columns it came from.
//   three warps issue loads, products and stores.
// V has three stages, as V' is wanted early and P V comes late in a chunk; o is staged in
// the stage it leaves and goes out by tensor stores (straight from registers, 16 or 32 bytes
// a row: 137 and 124 us).  Each role's loop is kept short, in rolled pieces of 32 columns:
// unrolled throughout, the roles' code pushed each other out of the instruction caches
// (2 x 8192 x 32 heads: 283 us against 126).
//
// Roundings to 16 bits: P and the operand copy of S, each at most half a step of
// the type, as o itself is.  The state proper stays in 32 bits in tensor memory, and what is added
// to it is V' in two pieces (hi + lo, within 3 2^-16 of v' in bf16, 2^-18 in the mean; in fp16 2^-21 of it, or
// 2^-36): one piece would put a 16-bit error into a 32-bit result that later calls build on.  fp16 has no
// room for the operands' ranges: the rows of P, the copy of S and the second piece of V' are scaled by
// powers of two to fit.
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
  // Warps 0-7 values and weights, 8-15 state and output, then loads, products, stores.
  static constexpr int THREADS = 19 * 32;
  static constexpr int W_TMA = 16, W_MMA = 17, W_STORE = 18;
  static constexpr int NV = 3;                    // stages of V
  // Tensor memory: chunk n's Q K^T at 128 (n & 1), P in the first 16 of every 32 columns
  // of it, Q S at 256, P V at 320, the state in two parts at 384 (what the second
  // piece of V' adds is kept apart, so that one product of 128 columns reads K once).
  static constexpr uint32_t TM_COLS = 512;
  __device__ static constexpr uint32_t tm_s(int b) { return 128u * b; }
  static constexpr uint32_t TM_QS = 256, TM_PV = 320, TM_STATE = 384, TM_SECOND = 64;  // (the second part, from the first)
};

template <int D>
struct LinearSmem {
  using C = LinearCfg<D>;
  alignas(1024) uint8_t q[2][C::TILE];
  alignas(1024) uint8_t k[2][C::TILE];
  alignas(1024) uint8_t v[C::NV][C::ATOM];
  alignas(1024) uint8_t vp[2][C::ATOM];  // V', first and second piece
  alignas(1024) uint8_t sb[D * 128];     // the state as an operand
  uint8_t row_max[2][2][128];  // fp16: the exponents of the largest scores in the two parts of a row
  int8_t row_scale[4][128];    // fp16: the powers of two that the rows of P were divided by,
  int state_scale[4];          // and the state (read up to two chunks late)
  float col[32];            // [j]: w^(31 - j)
  // Rows of the diagonal block: w^(lane - j), 0 where j > lane, for j = 0 .. 31 is
  // d[31 - lane + j] with d[m] = w^(31 - m) or 0.  Four copies, the c-th shifted by c, so that every
  // lane reads 16 aligned bytes; 72 floats apart, so that 8 lanes meet no bank twice.
  float diag[4][72];
  uint64_t qk_full[2], k_empty[2], q_empty[2], v_full[C::NV], v_empty[C::NV];
  uint64_t s_full[2], p_full[2];
  uint64_t stage_full[C::NV];
  uint64_t o_full, o_empty, ready, init, kv_done, teardown;
  uint32_t tmem_base;
  uint32_t part[2][8];
  int abort_flag;
};

// w^n for n >= 0 from log2 w (w = 0: 1, 0, 0, ...).
__device__ __forceinline__ float decay_pow(float log2w, int n) { return n == 0 ? 1.0f : exp2f(log2w * n); }

// fp16 operands are scaled by powers of two: the biased exponent of the largest
// magnitude m gives e such that m 2^-e is below 2^top (0, infinity and NaN: e = 0).
__device__ __forceinline__ int exponent_of(float m) { return static_cast<int>(__float_as_uint(m) >> 23); }
__device__ __forceinline__ int fit(int exponent, int top) {
  return exponent == 0 || exponent >= 255 ? 0 : max(-100, min(exponent - 126 - top, 120));
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// fp16: what the second piece of V' is multiplied by.  (It is at most half a step of the
// first one, 16: room for 2^11.)
constexpr float kSecondScale = 2048.0f;
// a -= kSecondScale x, for both fp16 halves of x.
__device__ __forceinline__ void subtract_scaled(uint32_t x, float& a0, float& a1) {
  asm("{\n .reg .b16 x0, x1, m;\n mov.b32 {x0, x1}, %2;\n mov.b16 m, 0xe800;\n"
      " fma.rn.f32.f16 %0, x0, m, %0;\n fma.rn.f32.f16 %1, x1, m, %1;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "r"(x));
}

template <int D, bool BF16, bool STATES>
__global__ void __launch_bounds__(LinearCfg<D>::THREADS, 1) linear_chunk_kernel(const __grid_constant__ LinearParams p) {
  using C = LinearCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  LinearSmem<D>& sm = *reinterpret_cast<LinearSmem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = blockIdx.x, h = blockIdx.y, place = blockIdx.z / p.segs, seg = blockIdx.z - place * p.segs;

  pdl_launch_dependents();
  pdl_wait();
  if (smem_u32(smem_raw) & 1023u) {  // (the swizzled tiles need it; there is no room to round up)
    if (tid == 0 && p.err) atomicOr(p.err, 1u << kErrLinearTeardown);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.qk_full[i], STATES ? 1 : 2);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 256);
    }
    for (int i = 0; i < C::NV; ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.stage_full[i], 256);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, 256);
    mbar_init(&sm.ready, STATES ? 256 : 512);  // V', and (not STATES) S as an operand and decayed
    mbar_init(&sm.init, 256);                  // (STATES) the state the segment (by_chunk: the chunk) starts from
    mbar_init(&sm.kv_done, 1);
    mbar_init(&sm.teardown, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  int b = place;
  if (p.longest_first) {
    // CTAs start in the order of blockIdx: the place-th longest sequence is this one's.
    int* lens = reinterpret_cast<int*>(sm.sb);
    int row, mine = 0;
    if (tid < p.B) {
      sequence_rows(p, tid, row, mine);
      lens[tid] = mine;
    }
    __syncthreads();
    if (tid < p.B) {
      int rank = 0;
      for (int i = 0; i < p.B; ++i) rank += lens[i] > mine || (lens[i] == mine && i < tid);
      if (rank == place) lens[kLongestFirst] = tid;
    }
    __syncthreads();
    b = lens[kLongestFirst];
    __syncthreads();
  }
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
  const bool grows = log2w > 0.0f;
  // fp16 has no room for weights above 1: those of V' are then taken back to the chunk's start.
  const bool back = !BF16 && grows;
  // Decays above 1 leave fp32 over a segment, so that the first launch carries them from chunk
  // to chunk as the second does.
  const bool by_chunk = !STATES || grows;
  if (tid < 32) sm.col[tid] = decay_pow(log2w, 31 - tid);
  if (tid >= 64 && tid < 64 + 4 * 72) {
    const int c = (tid - 64) / 72, m = (tid - 64) % 72 + c;
    sm.diag[c][m - c] = m <= 31 ? decay_pow(log2w, 31 - m) : 0.0f;
  }
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
        const int s = n & 1, sv = n % C::NV;
        // (K is free once K^T V' is done, Q after Q S.)
        if (!(ok = w.wait(&sm.k_empty[s], ((n >> 1) & 1) ^ 1, kErrLinearWait))) break;
        mbar_arrive_expect_tx(&sm.qk_full[s], C::TILE);
        ++qk_armed;
#pragma unroll
        for (int c = 0; c < C::NCHUNK; ++c)
          tma_load_4d(sm.k[s] + c * C::ATOM, &p.tm_k, &sm.qk_full[s], c * 64, row_of(n), hk, bc);
        if constexpr (!STATES) {
          if (!(ok = w.wait(&sm.q_empty[s], ((n >> 1) & 1) ^ 1, kErrLinearWait))) break;
          mbar_arrive_expect_tx(&sm.qk_full[s], C::TILE);
#pragma unroll
          for (int c = 0; c < C::NCHUNK; ++c)
            tma_load_4d(sm.q[s] + c * C::ATOM, &p.tm_q, &sm.qk_full[s], c * 64, row_of(n), h, bc);
        }
        if (!(ok = w.wait(&sm.v_empty[sv], ((n / C::NV) & 1) ^ 1, kErrLinearWait))) break;
        mbar_arrive_expect_tx(&sm.v_full[sv], C::ATOM);
        ++v_armed;
        tma_load_4d(sm.v[sv], &p.tm_v, &sm.v_full[sv], half * C::N, row_of(n), hk, bc);
      }
      if (w.aborted()) {  // every copy started must land before shared memory is released
        const uint64_t dl = globaltimer_ns() + 50000000ull;
        for (int i = max(0, qk_armed - 2); i < qk_armed; ++i) wait_raw(&sm.qk_full[i & 1], (i >> 1) & 1, dl);
        for (int i = max(0, v_armed - C::NV); i < v_armed; ++i)
          wait_raw(&sm.v_full[i % C::NV], (i / C::NV) & 1, dl);
      }
    }
  } else if (warp == C::W_MMA) {
    // ===================== products (whole warp, one lane issues) ==============
    const uint32_t lead = elect_one() ? 1u : 0u;
    constexpr uint32_t id_s = idesc_f16_f32(BF16, 128, 128, false, false);
    constexpr uint32_t id_pv = idesc_f16_f32(BF16, 128, 64, false, true);
    constexpr uint32_t id_kv = idesc_f16_f32(BF16, 128, 128, true, true);
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
    // A chunk that the sequence ends in is multiplied once its rows behind the end have been
    // cleared (with V'): what they held may be NaN, and the weights there are 0.
    const int partial = (t1 - t0) % C::C != 0 ? chunks - 1 : -1;
    if (!STATES && chunks > 0) {
      ok = w.wait(&sm.qk_full[0], 0, kErrLinearWait);
      if (ok && partial == 0) ok = w.wait(&sm.ready, 0, kErrLinearWait);
      tc_fence_after();
      if (ok) issue_s(0);
    }
    for (int n = 0; ok && n < chunks; ++n) {
      const int s = n & 1;
      // S += K^T V'
      if (!(ok = w.wait(&sm.ready, n & 1, kErrLinearWait))) break;
      if (STATES && (n == 0 || grows) && !(ok = w.wait(&sm.init, n & 1, kErrLinearWait))) break;
      if (STATES && !(ok = w.wait(&sm.qk_full[s], (n >> 1) & 1, kErrLinearWait))) break;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < C::C / 16; ++i) {
        const uint64_t ka = ktd0 + static_cast<uint64_t>(s * (C::TILE >> 4) + ((i * 16 * 128) >> 4));
        umma_ss_warp(tmem + C::TM_STATE, ka, vpd0 + ((i * 16 * 128) >> 4), id_kv, 1u, lead);
      }
      umma_commit_warp(&sm.kv_done, lead);
      if constexpr (STATES) {
        umma_commit_warp(&sm.k_empty[s], lead);
        umma_commit_warp(&sm.v_empty[n % C::NV], lead);
      } else {
        umma_commit_warp(&sm.k_empty[s], lead);
        // Q S, once the o of the chunk before has been read
        if (n > 0) {
          if (!(ok = w.wait(&sm.o_empty, (n - 1) & 1, kErrLinearWait))) break;
          tc_fence_after();
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          umma_ss_warp(tmem + C::TM_QS, qd0 + static_cast<uint64_t>(s * (C::TILE >> 4) + (((i >> 2) * C::ATOM + (i & 3) * 32) >> 4)),
                       sbd + ((i * 16 * 128) >> 4), id_pv, i > 0 ? 1u : 0u, lead);
        umma_commit_warp(&sm.q_empty[s], lead);
        if (n + 1 < chunks) {
          if (!(ok = w.wait(&sm.qk_full[s ^ 1], ((n + 1) >> 1) & 1, kErrLinearWait))) break;
          if (n + 1 == partial && !(ok = w.wait(&sm.ready, (n + 1) & 1, kErrLinearWait))) break;
          tc_fence_after();
          issue_s(n + 1);  // (over the P whose P V was issued before)
        }
        // P V
        if (!(ok = w.wait(&sm.p_full[s], (n >> 1) & 1, kErrLinearWait))) break;
        tc_fence_after();
        const uint64_t vd = vd0 + static_cast<uint64_t>((n % C::NV) * (C::ATOM >> 4));
#pragma unroll
        for (int i = 0; i < C::C / 16; ++i)
          umma_ts_warp(tmem + C::TM_PV, tmem + C::tm_s(s) + 32 * (i >> 1) + 8 * (i & 1), vd + ((i * 16 * 128) >> 4), id_pv,
                       i > 0 ? 1u : 0u, lead);
        umma_commit_warp(&sm.o_full, lead);
      }
    }
    if constexpr (STATES) umma_commit_warp(&sm.o_full, lead);  // the segment's state is complete
    // All products must be done before tensor memory is freed.
    umma_commit_warp(&sm.teardown, lead);
    if (!wait_raw(&sm.teardown, 0, globaltimer_ns() + 50000000ull) && p.err) atomicOr(p.err, 1u << kErrLinearTeardown);
  } else if (warp == C::W_STORE) {
    // ===================== stores of whole chunks ================================
    if (!STATES && lane == 0) {
      for (int n = 0; n < chunks && t0 + (n + 1) * C::C <= t1; ++n) {
        // (One barrier per stage: a slow store may fall chunks behind, but a stage is not
        // filled again before it has been released here.)
        if (!w.wait(&sm.stage_full[n % C::NV], (n / C::NV) & 1, kErrLinearWait)) break;
        tma_store_4d(&p.tm_o, sm.v[n % C::NV], half * C::N, row0 + t0 + n * C::C, h, bc);
        bulk_commit();
        bulk_wait_read();
        mbar_arrive(&sm.v_empty[n % C::NV]);
      }
      bulk_wait_all();  // every store has completed before the CTA ends
    }
  } else if (warp < 8) {
    // ===================== values and weights =====================================
    const int part = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const float full = back ? decay_pow(-log2w, r + 1) : decay_pow(log2w, C::C - 1 - r);
    const float* diag = &sm.diag[(31 - lane) & 3][(31 - lane) & ~3];
    bool ok = true;
    // V' = w^(tokens behind it) v: up to where the state is wanted, the chunk's end and in
    // the first launch the segment's; with `back` w^-(tokens up to it) v, and the state is multiplied
    // by w^(tokens of the chunk) when it is read.  Thread = token r, 32 columns.  In packed 16-bit
    // arithmetic: with the weight f = f1 + f2 in two pieces, hi = f1 v rounded, f1 v - hi is exact
    // (a product of two significands less its upper half), and lo = that + f2 v, at most 2^-7 of v' in
    // bf16, where its rounding is at most 2^-15 of v' and f2's 2^-16.  fp16 has not the exponents for that: v' in 32 bits,
    // hi rounded from it, and lo = v' - hi, which is exact there, at 2^11 of its size: rounded to 2^-22
    // of v', or among the subnormal numbers to 2^-36 (2 x 8192 tokens of 32 heads: 118 us with a lo
    // of its own size, whose error is 2^-24 however small v is, 130 with this one).
    auto values = [&](int n) {
      const int sv = n % C::NV;
      ok = __all_sync(0xffffffffu, w.wait(&sm.v_full[sv], (n / C::NV) & 1, kErrLinearWait));
      if (!ok) return;
      const int left = t1 - t0 - n * C::C;  // tokens from this chunk on
      const int live = min(left, C::C);
      const float f = r >= live                            ? 0.0f
                      : back || (by_chunk && live == C::C) ? full
                                                           : decay_pow(log2w, (by_chunk ? live : left) - 1 - r);
      uint8_t* src = sm.v[sv] + r * 128;
      uint32_t hi[16], lo[16];
      float f1, unused;
      const uint32_t fw = pack_bf16(f, f);
      unpack16<true>(fw, f1, unused);
      const uint32_t gw = pack_bf16(f - f1, f - f1);
      const uint64_t weight = f2_pack(f, f), up = f2_pack(f * kSecondScale, f * kSecondScale);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + (((4 * part + i) ^ (r & 7)) << 4));
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t v2 = r < live ? in[e] : 0u;  // (rows of nobody may hold anything)
          uint32_t &first = hi[4 * i + e], &second = lo[4 * i + e];
          if constexpr (BF16) {
            first = mul_bf16x2(v2, fw);
            second = fma_bf16x2(v2, gw, fma_bf16x2(v2, fw, first ^ 0x80008000u));
          } else {
            float x, y;
            unpack16<BF16>(v2, x, y);
            const uint64_t both = f2_pack(x, y);
            f2_unpack(f2_mul(both, weight), x, y);
            first = pack16<BF16>(x, y);
            f2_unpack(f2_mul(both, up), x, y);
            subtract_scaled(first, x, y);
            second = pack16<BF16>(x, y);
          }
        }
      }
      if (live < C::C) {
        // What lies behind the end meets weights of 0, and 0 * NaN is not 0.  (Q K^T of
        // this chunk waits for it too.)
        ok = __all_sync(0xffffffffu, w.wait(&sm.qk_full[n & 1], (n >> 1) & 1, kErrLinearWait));
        if (!ok) return;
        if (r >= live) {
#pragma unroll 1
          for (int i = 4 * part; i < 4 * part + 4; ++i) {
            const int at = (i ^ (r & 7)) << 4;
            *reinterpret_cast<uint4*>(src + at) = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < C::NCHUNK; ++c)
              *reinterpret_cast<uint4*>(sm.k[n & 1] + c * C::ATOM + r * 128 + at) = make_uint4(0, 0, 0, 0);
          }
        }
      }
      if (n > 0) ok = __all_sync(0xffffffffu, w.wait(&sm.kv_done, (n - 1) & 1, kErrLinearWait));
      if (!ok) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = r * 128 + (((4 * part + i) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(sm.vp[0] + at) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
        *reinterpret_cast<uint4*>(sm.vp[1] + at) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(&sm.ready);
    };
    // The decay from the last token of block cb down to row r, right of it.
    auto row_decay = [&](int cb) { return exp2f(log2w * (lane + 1 + 32 * (wq - 1 - cb))); };
    // P_ij = scale w^(i-j) q_i . k_j in blocks of 32 columns, thread = row i = r: blocks part
    // and part + 2, of which those right of the diagonal one are 0.  False: all threads that
    // share a barrier leave.
    auto weights = [&](int n) -> bool {
      if (ok) ok = __all_sync(0xffffffffu, w.wait(&sm.s_full[n & 1], (n >> 1) & 1, kErrLinearWait));
      if (BF16 && !ok) return false;
      tc_fence_after();
      const uint32_t base = tmem + C::tm_s(n & 1) + lanes;
      float f = p.scale;
      if constexpr (!BF16) {
        // fp16: the row's largest score decides a power of two that fits its weights (at
        // most 2^11, and 2^35 below for the small).  Decays above 1 make any multiple of a
        // score: then the scores of 16 columns at a time count with the largest decay there (at
        // most w^15 more than their own; below 2^15, so that the largest weight lies above w^-15 2^14).
        float m = 0.0f;
        if (ok) {
#pragma unroll 1
          for (int cb = part; cb <= wq; cb += 2) {
            uint32_t x[32];
            tmem_ld32(base + 32 * cb, x);
            tmem_ld_wait();
            reg_fence(x);
            if (cb == wq) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = j <= lane ? x[j] : 0u;
            }
            float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              m0 = fmax3(m0, fabsf(__uint_as_float(x[j])), fabsf(__uint_as_float(x[j + 1])));
              m1 = fmax3(m1, fabsf(__uint_as_float(x[j + 16])), fabsf(__uint_as_float(x[j + 17])));
            }
            if (grows) {
              const float* c = cb < wq ? sm.col : diag;
              const float down = cb < wq ? row_decay(cb) : 1.0f;
              m0 *= c[0] * down;
              m1 *= c[16] * down;
            }
            m = fmax3(m, m0, m1);
          }
        }
        sm.row_max[n & 1][part][r] = static_cast<uint8_t>(exponent_of(m * p.scale));
        // (The two warps of a row come here, aborted or not, and leave together.)
        ok = !named_bar_or(2 + wq, 64, !ok);
        if (!ok) return false;
        const int e = fit(max(sm.row_max[n & 1][0][r], sm.row_max[n & 1][1][r]), grows ? 15 : 11);
        if (part == 0) sm.row_scale[n & 3][r] = static_cast<int8_t>(e);
        f *= two_to(-e);
      }
#pragma unroll 1
      for (int cb = part; cb < 4; cb += 2) {
        uint32_t pk[16];
        if (cb > wq) {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = 0u;
        } else {
          uint32_t x[32];
          tmem_ld32(base + 32 * cb, x);
          // w^(i-j): left of the diagonal block the row's power down to the block's last
          // column times the column's from there, in it the table's.
          const float rowf = cb < wq ? f * row_decay(cb) : f;
          const float4* c4 = reinterpret_cast<const float4*>(cb < wq ? sm.col : diag);
          const uint64_t f2 = f2_pack(rowf, rowf);
          tmem_ld_wait();
          reg_fence(x);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 c = c4[j / 4];
            float x0, x1, x2, x3;
            f2_unpack(f2_mul(f2_mul(f2_pack(c.x, c.y), f2), f2_pack(__uint_as_float(x[j]), __uint_as_float(x[j + 1]))),
                      x0, x1);
            f2_unpack(f2_mul(f2_mul(f2_pack(c.z, c.w), f2), f2_pack(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]))),
                      x2, x3);
            pk[j / 2] = pack16<BF16>(x0, x1);
            pk[j / 2 + 1] = pack16<BF16>(x2, x3);
          }
        }
        tmem_st16(base + 32 * cb, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sm.p_full[n & 1]);
      return true;
    };
#pragma unroll 1
    for (int n = 0; n < chunks; ++n) {
      values(n);
      if constexpr (STATES) {
        if (!ok) break;
      } else {
        if (!weights(n)) break;
      }
    }
  } else if (warp < 16) {
    // ===================== state and output ======================================
    // Thread = row of S and of o, and 32 of its columns.
    const int part = (warp - 8) >> 2, wq = warp & 3, r = wq * 32 + lane, col = 32 * part;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t at = tmem + C::TM_STATE + col + lanes;
    // (d = 64: rows 64 .. 127 of tensor memory repeat rows 0 .. 63, and are worked on alike,
    // but only the first are written.)
    const bool mine = D == 128 || wq < 2;
    const int64_t state_at = (static_cast<int64_t>(slot) * p.Hq + h) * head + half * C::N + (r % D) * D + col;
    const int64_t row_at = work_at + (r % D) * D + col;
    bool ok = true;
    // Waits until the products so far are in S.
    auto reach = [&](uint64_t* bar, int phase) {
      ok = __all_sync(0xffffffffu, w.wait(bar, phase & 1, kErrLinearWait));
      tc_fence_after();
    };
    {
      // The state before the first token: state_in, or the states of the segments before
      // this one, decayed up to here.
      float s[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = 0.0f;
      auto add = [&](const float* from, float f) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 x = *reinterpret_cast<const float4*>(from + i);
          s[i] = fmaf(x.x, f, s[i]);
          s[i + 1] = fmaf(x.y, f, s[i + 1]);
          s[i + 2] = fmaf(x.z, f, s[i + 2]);
          s[i + 3] = fmaf(x.w, f, s[i + 3]);
        }
      };
      {
        float* copy = p.work + (p.segs - 1) * work_seg + row_at;
        if (seg == 0 && p.state_in != nullptr && slot >= 0) {
          // (Cut sequences: state_out may be state_in, whose last segment may be done before
          // this one starts: it is read from where the first launch has put it.)
          add(STATES || last ? p.state_in + state_at : copy, 1.0f);
          if (STATES && mine)
#pragma unroll
            for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(copy + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
        } else if (!STATES && seg > 0 && grows) {
          // (w^seg_len in steps that fp32 holds: what is 0 stays 0, whatever it is.)
          const float e = log2w * seg_len;
#pragma unroll 1
          for (int i = 0; i < seg; ++i) {
#pragma unroll 1
            for (int j = 0; i > 0 && j < 3; ++j) {
              const float f = exp2f(fminf(fmaxf(e - 126.0f * j, 0.0f), 126.0f));
#pragma unroll
              for (int x = 0; x < 32; ++x) s[x] *= f;
            }
            add(p.work + i * work_seg + row_at, 1.0f);
          }
        } else if (!STATES && seg > 0) {
#pragma unroll 1
          for (int i = seg - 1; i >= 0; --i) {
            const float f = decay_pow(log2w, (seg - 1 - i) * seg_len);
            if (f == 0.0f) break;
            add(p.work + i * work_seg + row_at, f);
          }
        }
        __syncwarp();
        const float f = by_chunk ? 1.0f : decay_pow(log2w, t1 - t0);
        uint32_t a[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] = __float_as_uint(s[j] * f);
        tmem_st32(at, a);
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] = 0u;
        tmem_st32(at + C::TM_SECOND, a);
        tmem_st_wait();
      }
    }
    // Both parts of S (with `back`, before the decays of the chunk that was added last).
    auto read = [&](uint32_t (&a)[32]) {
      uint32_t c[32];
      tmem_ld32(at, a);
      tmem_ld32(at + C::TM_SECOND, c);
      tmem_ld_wait();
      reg_fence(a);
      reg_fence(c);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float x, y;
        const uint64_t first = f2_pack(__uint_as_float(a[j]), __uint_as_float(a[j + 1]));
        const uint64_t second = f2_pack(__uint_as_float(c[j]), __uint_as_float(c[j + 1]));
        f2_unpack(BF16 ? f2_add(first, second) : f2_fma(second, f2_pack(1.0f / kSecondScale, 1.0f / kSecondScale), first),
                  x, y);
        a[j] = __float_as_uint(x);
        a[j + 1] = __float_as_uint(y);
      }
    };
    auto clear2 = [&] {  // the second part of S
      const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 32; j += 8) tmem_st8(at + C::TM_SECOND + j, z);
    };
    auto finish = [&](float* to) {  // S to memory
      uint32_t a[32];
      read(a);
      if (!mine) return;
      if (back) {
        const float f = chunks > 0 ? decay_pow(log2w, t1 - t0 - (chunks - 1) * C::C) : 1.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) * f);
      }
#pragma unroll
      for (int j = 0; j < 32; j += 4) *reinterpret_cast<uint4*>(to + j) = make_uint4(a[j], a[j + 1], a[j + 2], a[j + 3]);
    };
    if constexpr (STATES) {
#pragma unroll 1
      for (int n = 0; n < (grows ? chunks : 1); ++n) {
        if (grows) {
          if (n > 0) reach(&sm.kv_done, n - 1);
          if (!ok) break;
          uint32_t a[32];
          read(a);
          // (Chunks of this launch are whole.)
          const float f = back && n == 0 ? 1.0f : decay_pow(log2w, C::C);
#pragma unroll
          for (int j = 0; j < 32; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) * f);
          tmem_st32(at, a);
          clear2();
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&sm.init);
      }
      if (ok) reach(&sm.o_full, 0);
      if (ok) finish(p.work + seg * work_seg + row_at);
    } else {
      const float full = decay_pow(log2w, C::C), since = p.scale * decay_pow(log2w, r + 1);
      uint8_t* sb_row = sm.sb + r * 128;
      uint16_t* out = static_cast<uint16_t*>(p.o) + bc * p.o_batch + h * p.o_head + half * C::N + col;
      // False: all threads that share a barrier leave.
      auto state = [&](int n) -> bool {
        if (ok && n > 0) reach(&sm.kv_done, n - 1);
        uint32_t a[32];
        if (ok) read(a);
        const float since_read = back && n > 0 ? full : 1.0f;
        float down = 1.0f;
        if constexpr (!BF16) {
          // fp16: one power of two for the whole operand, its largest element below 2^15.
          float m = 0.0f;
          if (ok)
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              m = fmax3(m, fabsf(__uint_as_float(a[j])), fabsf(__uint_as_float(a[j + 1])));
          const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(m * since_read));
          if (lane == 0) sm.part[n & 1][warp - 8] = top;
          // (Every thread comes here, aborted or not, and all leave together.)
          ok = !named_bar_or(1, 256, !ok);
          uint32_t all = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) all = max(all, sm.part[n & 1][i]);
          const int e = fit(exponent_of(__uint_as_float(all)), 15);
          if (warp == 8 && lane == 0) sm.state_scale[n & 3] = e;
          down = two_to(-e) * since_read;
        }
        if (!ok) return false;
        // (Q S of the chunk before has read the operand.)
        if (n > 0) ok = __all_sync(0xffffffffu, w.wait(&sm.q_empty[(n - 1) & 1], ((n - 1) >> 1) & 1, kErrLinearWait));
        if (!ok) return !BF16;
        const int m = t1 - t0 - n * C::C;
        const float f = back ? since_read : m >= C::C ? full : decay_pow(log2w, m);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo = __uint_as_float(a[8 * j + 2 * e]), hi = __uint_as_float(a[8 * j + 2 * e + 1]);
            if constexpr (!BF16) lo *= down, hi *= down;
            x[e] = pack16<BF16>(lo, hi);
          }
          if (mine) *reinterpret_cast<uint4*>(sb_row + (((4 * part + j) ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
        }
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float x, y;
          f2_unpack(f2_mul(f2_pack(__uint_as_float(a[j]), __uint_as_float(a[j + 1])), f2_pack(f, f)), x, y);
          a[j] = __float_as_uint(x);
          a[j + 1] = __float_as_uint(y);
        }
        tmem_st32(at, a);
        clear2();
        tmem_st_wait();
        tc_fence_before();
        fence_proxy_async_smem();
        mbar_arrive(&sm.ready);
        return true;
      };
      auto output = [&](int n) {
        reach(&sm.o_full, n);
        if (!ok) return;
        float fi = 1.0f, fs = since;
        if constexpr (!BF16) {
          fi = two_to(sm.row_scale[n & 3][r]);
          fs *= two_to(sm.state_scale[n & 3]);
        }
        uint32_t a[32], x[32];
        tmem_ld32(tmem + C::TM_PV + col + lanes, a);
        tmem_ld32(tmem + C::TM_QS + col + lanes, x);
        tmem_ld_wait();
        reg_fence(a);
        reg_fence(x);
        tc_fence_before();
        mbar_arrive(&sm.o_empty);
        // (P V was the last to read the chunk's V.  128-byte swizzle, as the tensor store reads.)
        uint8_t* stage = sm.v[n % C::NV];
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
          *reinterpret_cast<uint4*>(stage + r * 128 + (((4 * part + i) ^ (r & 7)) << 4)) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (t0 + (n + 1) * C::C <= t1) {
          fence_proxy_async_smem();  // the tensor store, and the next load of V, come after these
          mbar_arrive(&sm.stage_full[n % C::NV]);
          return;
        }
        // The last chunk, cut by the sequence's end: row by row, 8 x 64 bytes at a time.
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int row = wq * 32 + 8 * i + (lane >> 2), q = lane & 3, t = t0 + n * C::C + row;
          if (t < t1)
            *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row0 + t) * p.o_row + q * 8) =
                *reinterpret_cast<const uint4*>(stage + row * 128 + (((4 * part + q) ^ (row & 7)) << 4));
        }
      };
#pragma unroll 1
      for (int n = 0; n <= chunks; ++n) {
        if (n < chunks && !state(n)) break;
        if (ok && n > 0) output(n - 1);
        if (BF16 && !ok) break;
      }
      if (ok && last && chunks > 0) reach(&sm.kv_done, chunks - 1);
      if (ok && last && p.state_out != nullptr && slot >= 0) finish(p.state_out + state_at);
    }
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
  constexpr size_t smem = sizeof(LinearSmem<D>);
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
