// linear.h -- parameters of linear attention with a decay per head, and what its
// kernels share.
#pragma once
#include "../../include/attn_fwd.h"
#include "common.cuh"

namespace attn {

struct LinearParams {
  const void *q, *k, *v;
  void* o;
  const float* log_decay;
  const float* state_in;   // [num_states][Hq][d][d] or nullptr: zeros
  float* state_out;        // likewise, or nullptr: not kept
  const int32_t* index;    // [B] rows of both, or nullptr: b
  const int32_t* cu;       // packed sequences: [B + 1]; nullptr: dense, L rows each
  int num_states, Hq, group, L, total;
  attn_strides sq, sk, sv, so;
  float scale;
  unsigned int* err;
};

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
__device__ __forceinline__ void sequence_rows(const LinearParams& p, int b, int64_t& row0, int& len) {
  row0 = 0;
  len = p.L;
  if (p.cu != nullptr) {
    const int first = p.cu[b], last = p.cu[b + 1];
    row0 = first;
    len = first < 0 || first > p.total ? 0 : max(0, min(last, p.total) - first);
  }
}

}  // namespace attn
