// softmax.cuh -- row arithmetic of the online softmax shared by the prefill and
// tree kernels (one thread per query row, its scores in registers).
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace attn {

// Maximum of N values: a tree of 3-input max instructions (N = 128: 64
// instructions, depth 5).
template <int N>
__device__ __forceinline__ float max_n(const float* v) {
  if constexpr (N == 1) {
    return v[0];
  } else if constexpr (N == 2) {
    return fmaxf(v[0], v[1]);
  } else if constexpr (N == 3) {
    return fmax3(v[0], v[1], v[2]);
  } else {
    constexpr int M = (N + 2) / 3;
    float m[M];
#pragma unroll
    for (int i = 0; i < M; ++i)
      m[i] = 3 * i + 2 < N ? fmax3(v[3 * i], v[3 * i + 1], v[3 * i + 2])
                           : (3 * i + 1 < N ? fmaxf(v[3 * i], v[3 * i + 1]) : v[3 * i]);
    return max_n<M>(m);
  }
}

// P for one row: p_c = 2^(s_c * a - b) for c < 2 NP (a = scale*log2e, or
// cap*log2e when s holds tanh values), the FMA done two lanes at a time,
// packed to bf16/fp16 pairs, with 4 packed partial sums (8 lanes).  A masked
// score is -inf and gives p = 0 exactly.
template <bool BF16, int NP, int I = 0>
__device__ __forceinline__ void exp_pack_row(const float* s, uint64_t a2, uint64_t nb2,
                                             uint32_t* pk, uint64_t* acc2) {
  if constexpr (I < NP) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(s[2 * I], s[2 * I + 1]), a2, nb2), x0, x1);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    acc2[I & 3] = f2_add(acc2[I & 3], f2_pack(p0, p1));
    pk[I] = BF16 ? pack_bf16(p0, p1) : pack_f16(p0, p1);
    exp_pack_row<BF16, NP, I + 1>(s, a2, nb2, pk, acc2);
  }
}

// Soft-cap in the form the softmax consumes: s <- r = 1 / (2^(2 y log2 e) + 1)
// with y = in_scale * s, so that tanh(y) = 1 - 2 r and the capped score in
// log2 units is c (1 - 2 r), c = cap * log2 e.  The exponent's FMA then takes
// r directly (r * (-2c) + (c - m)) and the row maximum is c (1 - 2 min r):
// the tanh's own final FMA disappears from the chain.
template <int N>
__device__ __forceinline__ void softcap_r_n(float* s, float in_scale) {
  const uint64_t k2 = f2_pack(in_scale * 2.0f * kLog2e, in_scale * 2.0f * kLog2e);
  const uint64_t one2 = f2_pack(1.0f, 1.0f);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float e0, e1;
    f2_unpack(f2_mul(f2_pack(s[2 * i], s[2 * i + 1]), k2), e0, e1);
    e0 = ex2_approx(e0);
    e1 = ex2_approx(e1);
    float d0, d1;
    f2_unpack(f2_add(f2_pack(e0, e1), one2), d0, d1);
    s[2 * i] = rcp_approx(d0);
    s[2 * i + 1] = rcp_approx(d1);
  }
}

// Minimum of N values (a tree of 3-input min instructions).
template <int N>
__device__ __forceinline__ float min_n(const float* v) {
  if constexpr (N == 1) {
    return v[0];
  } else if constexpr (N == 2) {
    return fminf(v[0], v[1]);
  } else if constexpr (N == 3) {
    return fmin3(v[0], v[1], v[2]);
  } else {
    constexpr int M = (N + 2) / 3;
    float m[M];
#pragma unroll
    for (int i = 0; i < M; ++i)
      m[i] = 3 * i + 2 < N ? fmin3(v[3 * i], v[3 * i + 1], v[3 * i + 2])
                           : (3 * i + 1 < N ? fminf(v[3 * i], v[3 * i + 1]) : v[3 * i]);
    return min_n<M>(m);
  }
}

// Wait for a barrier phase ignoring the abort flag (teardown only).
__device__ __forceinline__ bool wait_raw(uint64_t* bar, uint32_t parity, uint64_t deadline) {
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() > deadline) return false;
  }
  return true;
}

// The low n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

}  // namespace attn
