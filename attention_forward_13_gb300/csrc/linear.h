// linear.h -- parameters of linear attention with a decay per head, and what its
// kernels share.
#pragma once
#include "../../include/attn_fwd.h"
#include "common.cuh"

#include <initializer_list>

namespace attn {

constexpr int kLinearChunk = 128;  // tokens per chunk
constexpr int kLongestFirst = 128;  // sequences that every CTA ranks for itself

struct LinearParams {
  CUtensorMap tm_q, tm_k, tm_v, tm_o;  // 4-D (d, rows, heads, batch), box {64, 128, 1, 1}
  void* o;
  const float* log_decay;
  const float* state_in;   // [num_states][Hq][d][d] or nullptr: zeros
  float* state_out;        // likewise, or nullptr: not kept
  const int32_t* index;    // [B] rows of both, or nullptr: b
  const int32_t* cu;       // packed sequences: [B + 1]; nullptr: dense, L rows each
  float* work;             // [segs][B][Hq][d][d]: states of all segments but the last, then state_in
  int num_states, B, Hq, group, L, total;
  int segs, seg_chunks;    // pieces a sequence is cut into, chunks of each
  int longest_first;       // packed sequences in order of their lengths (B <= kLongestFirst)
  int64_t o_batch, o_head, o_row;
  float scale;
  unsigned int* err;
  uint64_t timeout_ns;
};

// Pieces along the sequence.  Heads and halves of 64 columns are a CTA each and walk
// the chunks in order; where they leave SMs idle, the walk is cut into segments,
// whose states are summed up first, in a launch of its own that reads k and v once
// more (and takes about half the time a chunk).  As many pieces as the longest walk is
// longer than an SM's share of all chunks, rounded down (16 heads of 2048 tokens, d = 128, bf16
// and fp16: 24.0 -> 22.7 and 33 -> 25.8 us; sequences of 3000, 200, 100 and 50 tokens, 16
// heads, d = 64: 37 -> 24 and 47 -> 27; rounded up, 16 sequences of 1 to 3001: 36 -> 58 and
// 47 -> 68).  Segments that short sequences do not
// have are CTAs as well, that leave at once: no more than eight for every SM.
inline void linear_segments(int B, int Hq, int max_len, int64_t total, int d, int* segs, int* seg_chunks) {
  constexpr int64_t kSms = 152;
  const int chunks = max_len / kLinearChunk + (max_len % kLinearChunk != 0 ? 1 : 0);
  const int64_t ctas = static_cast<int64_t>(B) * Hq * (d / 64), most = static_cast<int64_t>(B) * chunks;
  int64_t all = total / kLinearChunk + (B + 1) / 2;  // chunks of all sequences, about
  if (all > most) all = most;
  int64_t n = all > 0 ? chunks * kSms / (all * Hq * (d / 64)) : 1;
  for (const int64_t most_segs : {static_cast<int64_t>(chunks / 2), 8 * kSms / (ctas > 0 ? ctas : 1),
                                  static_cast<int64_t>(65535 / (B > 0 ? B : 1)), static_cast<int64_t>(16)})
    n = n < most_segs ? n : most_segs;
  n = n > 1 ? n : 1;
  const int per = chunks > 0 ? static_cast<int>((chunks + n - 1) / n) : 1;
  *seg_chunks = per;
  *segs = chunks > 0 ? (chunks + per - 1) / per : 1;
}

// The two launches (linear_d64.cu, linear_d128.cu).
template <int D>
cudaError_t launch_linear_d(const LinearParams& p, bool bf16, cudaStream_t stream);

// The state of sequence b, -1 for none.  Every thread of the block calls it.  A
// row that is out of range or an earlier sequence's is none, and an error.
__device__ __forceinline__ int state_of(const int32_t* index, int num_states, int b, unsigned int* err, bool tell) {
  if (index == nullptr) return b;
  const int slot = index[b];
  if (slot == -1) return -1;
  bool bad = slot < 0 || slot >= num_states;
  if (!bad)
    for (int i = threadIdx.x; i < b; i += blockDim.x) bad |= index[i] == slot;
  if (!__syncthreads_or(bad)) return slot;
  if (tell && threadIdx.x == 0 && err) atomicOr(err, 1u << kErrCacheBadIndex);
  return -1;
}

// First row and length of sequence b, never past the packed tensors whatever
// cu_seqlens holds.
__device__ __forceinline__ void sequence_rows(const LinearParams& p, int b, int& row0, int& len) {
  row0 = 0;
  len = p.L;
  if (p.cu != nullptr) {
    const int first = p.cu[b], last = p.cu[b + 1];
    // (Compared before they are subtracted: an end far below 0 would leave 32 bits.)
    row0 = first;
    len = first < 0 || last <= first || first >= p.total ? 0 : min(last, p.total) - first;
  }
}

}  // namespace attn
