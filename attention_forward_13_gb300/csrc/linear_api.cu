// linear_api.cu -- linear attention with a decay per head: the C entry points and
// the recurrent kernel for single tokens (include/attn_fwd.h states the rules).
#include "host.h"
#include "launch.h"
#include "linear.h"
#include "overlap.h"
#include "ptx.cuh"

#include <algorithm>
#include <cmath>

using namespace attn;

namespace {

// Rows of one call: no sum of a row and a segment leaves 32 bits.
constexpr int kLinearMaxRows = 1 << 30;

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t x) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
  return __half2float(*reinterpret_cast<const __half*>(&x));
}
template <bool BF16>
__device__ __forceinline__ uint16_t from_float(float x) {
  return static_cast<uint16_t>(BF16 ? pack_bf16(x, 0.0f) : pack_f16(x, 0.0f));
}

// ---------------------------------------------------------------------------
// One token: S <- e^g S + k v^T, o = scale q^T S.  Bound by the state, which is
// read and written once (d * d * 8 bytes a head, against 4 d^2 operations).  A CTA
// holds COLS columns of one head's state in registers: a thread 4 neighbouring
// columns of every (kThreads / (COLS / 4))-th row, all its loads in flight at
// once.  o sums over the rows: over a thread's own, then over the lanes, then over
// the warps, always in that order.  64 sequences of 32 heads, d = 128: 40.9 us, 6.6 TB/s
// (0.99 of a copy's rate); one of 16 heads 2.0 us.
constexpr int kStepThreads = 256;

struct StepParams {
  const void *q, *k, *v;
  void* o;
  const float* log_decay;
  float* state;
  const int32_t* index;
  int num_states, Hq, group;
  int64_t q_batch, q_head, k_batch, k_head, v_batch, v_head, o_batch, o_head;
  float scale;
  unsigned int* err;
};

template <int D, int COLS, bool BF16>
__global__ void __launch_bounds__(kStepThreads) linear_step_kernel(const StepParams p) {
  constexpr int LANES = COLS / 4, ROWS = kStepThreads / LANES, PASSES = D / ROWS;
  __shared__ float sq[D], sk[D];
  __shared__ float part[kStepThreads / 32][COLS];
  pdl_launch_dependents();
  pdl_wait();
  const int col0 = blockIdx.x * COLS, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int slot = state_of(p.index, p.num_states, b, p.err, blockIdx.x == 0 && h == 0);
  const int c = col0 + 4 * (tid % LANES), r0 = tid / LANES;
  float* state = slot < 0 ? nullptr : p.state + (static_cast<int64_t>(slot) * p.Hq + h) * D * D + c;
  float4 s[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i)
    s[i] = state == nullptr ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : *reinterpret_cast<const float4*>(state + (r0 + i * ROWS) * D);
  const int hk = h / p.group;
  if (tid < D)
    sq[tid] = to_float<BF16>((static_cast<const uint16_t*>(p.q) + b * p.q_batch + h * p.q_head)[tid]);
  else if (tid < 2 * D)
    sk[tid - D] = to_float<BF16>((static_cast<const uint16_t*>(p.k) + b * p.k_batch + hk * p.k_head)[tid - D]);
  const uint2 vw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.v) + b * p.v_batch + hk * p.v_head + c);
  const float v[4] = {to_float<BF16>(vw.x & 0xffff), to_float<BF16>(vw.x >> 16), to_float<BF16>(vw.y & 0xffff),
                      to_float<BF16>(vw.y >> 16)};
  const float decay = expf(p.log_decay[h]);
  __syncthreads();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const float k = sk[r0 + i * ROWS], q = sq[r0 + i * ROWS];
    s[i].x = fmaf(k, v[0], s[i].x * decay);
    s[i].y = fmaf(k, v[1], s[i].y * decay);
    s[i].z = fmaf(k, v[2], s[i].z * decay);
    s[i].w = fmaf(k, v[3], s[i].w * decay);
    a.x = fmaf(q, s[i].x, a.x);
    a.y = fmaf(q, s[i].y, a.y);
    a.z = fmaf(q, s[i].z, a.z);
    a.w = fmaf(q, s[i].w, a.w);
    if (state != nullptr) *reinterpret_cast<float4*>(state + (r0 + i * ROWS) * D) = s[i];
  }
#pragma unroll
  for (int m = LANES; m < 32; m <<= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, m);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, m);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, m);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, m);
  }
  if ((tid & 31) < LANES) *reinterpret_cast<float4*>(&part[tid >> 5][4 * (tid & 31)]) = a;
  __syncthreads();
  if (tid < COLS) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < kStepThreads / 32; ++w) x += part[w][tid];
    (static_cast<uint16_t*>(p.o) + b * p.o_batch + h * p.o_head + col0)[tid] = from_float<BF16>(x * p.scale);
  }
}

template <int D, int COLS>
cudaError_t launch_step(const StepParams& p, int B, bool bf16, cudaStream_t stream) {
  const dim3 grid(D / COLS, p.Hq, B);
  return bf16 ? launch_pdl(linear_step_kernel<D, COLS, true>, grid, kStepThreads, 0, stream, p)
              : launch_pdl(linear_step_kernel<D, COLS, false>, grid, kStepThreads, 0, stream, p);
}

// ---------------------------------------------------------------------------
bool strides_ok(const attn_strides& s, bool row, bool batch) {
  return s.head > 0 && s.head % 8 == 0 && (!row || (s.row > 0 && s.row % 8 == 0)) &&
         (!batch || (s.batch > 0 && s.batch % 8 == 0));
}

// Whether o shares memory with an input (CTAs of a head read what others have written).
bool over_inputs(const void* q, const void* k, const void* v, const void* o, const attn_strides& sq,
                 const attn_strides& sk, const attn_strides& sv, const attn_strides& so, int B, int Hq, int Hkv, int rows,
                 int d) {
  const Extent out{o, so, {B, Hq, rows}, d};
  return o == q || o == k || o == v || overlap(out, {q, sq, {B, Hq, rows}, d}) ||
         overlap(out, {k, sk, {B, Hkv, rows}, d}) || overlap(out, {v, sv, {B, Hkv, rows}, d});
}

// What all three entry points ask of their sizes, types and states.
attn_status check_common(const float* log_decay, const float* state_in, const float* state_out, const int32_t* index,
                         int num_states, int B, int Hq, int Hkv, int d, attn_dtype dtype, float scale) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || std::isnan(scale) || std::isinf(scale)) return ATTN_ERR_INVALID;
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return dtype == ATTN_E4M3 ? ATTN_ERR_UNSUPPORTED : ATTN_ERR_INVALID;
  if ((d != 64 && d != 128) || Hq > 65535 || B > 65535) return ATTN_ERR_UNSUPPORTED;
  if (B == 0) return ATTN_OK;
  if (log_decay == nullptr || !host_aligned(log_decay, 4) || !host_aligned(state_in, 16) ||
      !host_aligned(state_out, 16) || !host_aligned(index, 4))
    return ATTN_ERR_INVALID;
  if (state_in != nullptr || state_out != nullptr) {
    if (num_states <= 0 || (index == nullptr && num_states < B)) return ATTN_ERR_INVALID;
    // (One state is read while another is written: the same buffer, or two.)
    const uintptr_t in = reinterpret_cast<uintptr_t>(state_in), out = reinterpret_cast<uintptr_t>(state_out);
    const uint64_t bytes = sizeof(float) * static_cast<uint64_t>(num_states) * Hq * d * d;
    if (state_in != nullptr && state_out != nullptr && in != out && in < out + bytes && out < in + bytes)
      return ATTN_ERR_INVALID;
  }
  return ATTN_OK;
}

// Everything of a call of the chunked kernels that the dense and the packed form share:
// rows of a tensor (per batch), batches, the longest sequence.
attn_status linear_fwd(const void* q, const void* k, const void* v, void* o, const int32_t* cu, const float* log_decay,
                       const float* state_in, float* state_out, const int32_t* index, int num_states, int B, int rows,
                       int max_len, int Hq, int Hkv, int d, bool bf16, attn_strides sq, attn_strides sk,
                       attn_strides sv, attn_strides so, float scale, void* workspace, size_t workspace_bytes,
                       void* stream) {
  LinearParams p{};
  if (rows > 0) {
    for (const void* x : {q, k, v, static_cast<const void*>(o)})
      if (x == nullptr || !host_aligned(x, 16)) return ATTN_ERR_INVALID;
    const bool batches = cu == nullptr && B > 1;
    for (const attn_strides* s : {&sq, &sk, &sv, &so})
      if (!strides_ok(*s, true, batches)) return ATTN_ERR_INVALID;
    if (over_inputs(q, k, v, o, sq, sk, sv, so, cu == nullptr ? B : 1, Hq, Hkv, rows, d)) return ATTN_ERR_INVALID;
    const uint32_t box[4] = {64, kLinearChunk, 1, 1};
    auto map = [&](CUtensorMap* m, const void* base, const attn_strides& s, int heads) {
      const uint64_t dims[4] = {(uint64_t)d, (uint64_t)rows, (uint64_t)heads, cu != nullptr ? 1u : (uint64_t)B};
      const uint64_t st[3] = {(uint64_t)s.row * 2, (uint64_t)s.head * 2,
                              batches ? (uint64_t)s.batch * 2 : (uint64_t)s.head * 2};
      return host_make_map(m, base, bf16, 4, dims, st, box);
    };
    if (!map(&p.tm_q, q, sq, Hq) || !map(&p.tm_k, k, sk, Hkv) || !map(&p.tm_v, v, sv, Hkv) ||
        !map(&p.tm_o, o, so, Hq))
      return ATTN_ERR_INVALID;
  }
  const int64_t tokens = cu != nullptr ? rows : static_cast<int64_t>(B) * rows;
  linear_segments(B, Hq, max_len, tokens, d, &p.segs, &p.seg_chunks);
  const size_t need = attn_linear_workspace_bytes(B, Hq, max_len, tokens, d);
  if (need > 0 && (workspace == nullptr || !host_aligned(workspace, 16) || workspace_bytes < need))
    return ATTN_ERR_INVALID;
  p.o = o;
  p.cu = cu;
  p.log_decay = log_decay;
  p.state_in = state_in;
  p.state_out = state_out;
  p.index = state_in != nullptr || state_out != nullptr ? index : nullptr;
  p.work = static_cast<float*>(workspace);
  p.num_states = num_states;
  p.B = B;
  p.Hq = Hq;
  p.group = Hq / Hkv;
  // More CTAs than SMs, of different lengths: the long ones first, so that none is left
  // for the end (16 sequences up to 3001, 16 heads, d = 64: 36.2 us in bf16 and 47.2 in fp16, in
  // their own order 43.8 and 57).
  p.longest_first = cu != nullptr && B > 1 && B <= kLongestFirst && static_cast<int64_t>(B) * Hq * (d / 64) > 152;
  p.L = rows;
  p.total = rows;
  p.o_batch = so.batch;
  p.o_head = so.head;
  p.o_row = so.row;
  p.scale = scale > 0.0f ? scale : 1.0f / sqrtf(static_cast<float>(d));
  p.timeout_ns = host_timeout_ns();
  if (host_device_state(&p.err, nullptr) != ATTN_OK) return ATTN_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return host_finish(d == 64 ? launch_linear_d<64>(p, bf16, s) : launch_linear_d<128>(p, bf16, s),
                     p.segs > 1 ? "attn_linear_chunk_states+attn_linear_chunk" : "attn_linear_chunk");
}

}  // namespace

extern "C" {

size_t attn_linear_workspace_bytes(int B, int Hq, int max_seqlen, int64_t tokens, int d) {
  if (B <= 0 || Hq <= 0 || max_seqlen <= 0 || tokens < 0 || (d != 64 && d != 128)) return 0;
  int segs, chunks;
  linear_segments(B, Hq, max_seqlen, tokens, d, &segs, &chunks);
  return segs > 1 ? static_cast<size_t>(segs) * B * Hq * d * d * sizeof(float) : 0;
}

attn_status attn_linear_fwd(const void* q, const void* k, const void* v, void* o, const float* log_decay,
                            const float* state_in, float* state_out, const int32_t* state_index, int num_states,
                            int B, int Hq, int Hkv, int L, int d, attn_dtype dtype, attn_strides sq, attn_strides sk,
                            attn_strides sv, attn_strides so, float scale, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (L < 0) return ATTN_ERR_INVALID;
  const attn_status st =
      check_common(log_decay, state_in, state_out, state_index, num_states, B, Hq, Hkv, d, dtype, scale);
  if (st != ATTN_OK || B == 0) return st;
  if (L > kLinearMaxRows) return ATTN_ERR_UNSUPPORTED;
  return linear_fwd(q, k, v, o, nullptr, log_decay, state_in, state_out, state_index, num_states, B, L, L, Hq, Hkv, d,
                    dtype == ATTN_BF16, sq, sk, sv, so, scale, workspace, workspace_bytes, stream);
}

attn_status attn_linear_fwd_varlen(const void* q, const void* k, const void* v, void* o, const int32_t* cu_seqlens,
                                   const float* log_decay, const float* state_in, float* state_out,
                                   const int32_t* state_index, int num_states, int B, int total, int max_seqlen, int Hq,
                                   int Hkv, int d, attn_dtype dtype, attn_strides sq, attn_strides sk, attn_strides sv,
                                   attn_strides so, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (total < 0 || max_seqlen < 0) return ATTN_ERR_INVALID;
  const attn_status st =
      check_common(log_decay, state_in, state_out, state_index, num_states, B, Hq, Hkv, d, dtype, scale);
  if (st != ATTN_OK || B == 0) return st;
  if (cu_seqlens == nullptr || !host_aligned(cu_seqlens, 4)) return ATTN_ERR_INVALID;
  if (total > kLinearMaxRows || max_seqlen > kLinearMaxRows) return ATTN_ERR_UNSUPPORTED;
  return linear_fwd(q, k, v, o, cu_seqlens, log_decay, state_in, state_out, state_index, num_states, B, total, max_seqlen,
                    Hq, Hkv, d, dtype == ATTN_BF16, sq, sk, sv, so, scale, workspace, workspace_bytes, stream);
}

attn_status attn_linear_step(const void* q, const void* k, const void* v, void* o, const float* log_decay, float* state,
                             const int32_t* state_index, int num_states, int B, int Hq, int Hkv, int d, attn_dtype dtype,
                             attn_strides sq, attn_strides sk, attn_strides sv, attn_strides so, float scale,
                             void* stream) {
  const attn_status st = check_common(log_decay, state, state, state_index, num_states, B, Hq, Hkv, d, dtype, scale);
  if (st != ATTN_OK || B == 0) return st;
  for (const void* x : {q, k, v, static_cast<const void*>(o), static_cast<const void*>(state)})
    if (x == nullptr || !host_aligned(x, 16)) return ATTN_ERR_INVALID;
  for (const attn_strides* s : {&sq, &sk, &sv, &so})
    if (!strides_ok(*s, false, B > 1)) return ATTN_ERR_INVALID;
  if (over_inputs(q, k, v, o, sq, sk, sv, so, B, Hq, Hkv, 1, d)) return ATTN_ERR_INVALID;
  StepParams p{q, k, v, o, log_decay, state, state_index, num_states, Hq, Hq / Hkv,
               sq.batch, sq.head, sk.batch, sk.head, sv.batch, sv.head, so.batch, so.head,
               scale > 0.0f ? scale : 1.0f / sqrtf(static_cast<float>(d)), nullptr};
  int sms = 0;
  if (host_device_state(&p.err, &sms) != ATTN_OK) return ATTN_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Few heads leave SMs idle: their columns are dealt to several CTAs.
  const bool few = static_cast<int64_t>(B) * Hq < 2 * static_cast<int64_t>(sms);
  cudaError_t e;
  if (d == 64)
    e = few ? launch_step<64, 32>(p, B, dtype == ATTN_BF16, s) : launch_step<64, 64>(p, B, dtype == ATTN_BF16, s);
  else
    e = few ? launch_step<128, 32>(p, B, dtype == ATTN_BF16, s) : launch_step<128, 128>(p, B, dtype == ATTN_BF16, s);
  return host_finish(e, "attn_linear_step");
}

}  // extern "C"
