// launch.h -- host-side launchers of the kernels (one per translation unit),
// called by the C ABI layer in api.cu after validation.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include "common.cuh"

namespace attn {

// grid = number of CTAs; name receives the kernel's trait string.  xf is a
// ScoreXf value.  Dispatches to launch_prefill_d<64 / 128>.
// mask is a PrefillMask value.
cudaError_t launch_prefill(const PrefillKeepParams& p, int grid, int d, int dt, int mask,
                           int xf, cudaStream_t stream, char* name, size_t name_len);
// One per head dimension, each in its own translation unit (prefill_d64.cu,
// prefill_d128.cu) so the two compile in parallel.
// dt: PrefillDt (0 fp16, 1 bf16, 2 e4m3).
template <int D>
cudaError_t launch_prefill_d(const PrefillParams& p, int grid, int dt, bool masked, int xf,
                             cudaStream_t stream);
// The same for a window whose first tokens stay visible (prefill_keep_d64.cu,
// prefill_keep_d128.cu).
template <int D>
cudaError_t launch_prefill_keep_d(const PrefillKeepParams& p, int grid, int dt, int xf,
                                  cudaStream_t stream);

cudaError_t launch_decode(const DecodeParams& p, int d, bool bf16, bool softcap, int rows,
                          cudaStream_t stream, char* name, size_t name_len);
// feat: 0 none, 1 masks, 2 masks + ALiBi.  One per head dimension
// (decode_d64.cu, decode_d128.cu).
template <int D>
cudaError_t launch_decode_d(const DecodeParams& p, bool bf16, bool softcap, int feat,
                            cudaStream_t stream);

// One per head dimension (tree_d64.cu, tree_d128.cu).
template <int D>
cudaError_t launch_tree_d(const TreeParams& p, bool bf16, bool softcap, cudaStream_t stream);

cudaError_t launch_combine(const CombineParams& p, bool bf16, cudaStream_t stream, char* name,
                           size_t name_len);

// Launch with programmatic serialisation: the kernel may be set up while its
// predecessor in the stream still runs, and calls pdl_wait() before it touches
// global memory.
template <class... P, class... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The same for a kernel whose dynamic shared memory grows with the call, up to
// `most` bytes: the limit is raised to that once per device and never lowered, so
// that no call depends on the ones before it or on another host thread's.  (The
// 48 KB a block may have unasked count the kernel's own shared arrays too.)
template <auto kKern, class... A>
cudaError_t launch_pdl_upto(size_t most, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                            const A&... args) {
  static std::atomic<uint64_t> raised{0};  // bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(raised.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kKern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl(kKern, grid, threads, smem, stream, args...);
}

cudaError_t launch_selftest_timeout(unsigned int* err, unsigned long long timeout_ns,
                                    cudaStream_t stream);

}  // namespace attn
