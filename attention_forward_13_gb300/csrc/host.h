// host.h -- what the files of the C ABI layer share (defined in api.cu).
#pragma once
#include "../../include/attn_fwd.h"
#include "common.cuh"

namespace attn {

// The current device's error word and SM count.
attn_status host_device_state(unsigned int** err, int* num_sms);
// Tensor map with the 128-byte swizzle over a 16-bit tensor (make_map in api.cu).
bool host_make_map(CUtensorMap* m, const void* base, bool bf16, int rank, const uint64_t* dims,
                   const uint64_t* strides_bytes, const uint32_t* box);
// Options every attention entry point checks, and their resolved values.
attn_status host_check_opts(const attn_opts* opts, int Hq, bool allow_bias);
// Left bound of the window (negative: none) and the first tokens visible left of it.
int host_left(const attn_opts* opts);
int host_keep(const attn_opts* opts);
float host_scale(const attn_opts* opts, int d);
uint64_t host_timeout_ns();
// Records the kernel name of attn_last_kernel_name and turns a launch's
// result into a status.
attn_status host_finish(cudaError_t e, const char* name);

// Decode over a window with first tokens on the tree kernel (tree_api.cu): whether
// it has enough units to balance without cutting any, and the launch.  The
// arguments have been checked.
bool host_chain_applies(int B, int Lq, int Hq, int Hkv, int page_size, int max_pages, const attn_opts* opts);
attn_status host_chain(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
                       const int32_t* seqlens_k, void* o, float* lse, int B, int Lq, int Hq, int Hkv, int d,
                       bool bf16, int page_size, int num_pages, int max_pages, const attn_opts* opts,
                       cudaStream_t stream);

inline bool host_aligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace attn
