// tree_api.cu -- C ABI of the attention over a tree of drafted tokens: the tree's
// visibility masks and the entry point that checks and launches the attention
// kernels of tree_kernel.cuh.
#include "host.h"
#include "launch.h"
#include "ptx.cuh"

#include <cstdio>
#include <cstring>

using namespace attn;

namespace {

// Masks and depths from parent indices, one CTA per sequence, by pointer
// jumping in shared memory: with mask_i the bits of the ancestors passed so far
// and j_i the first one not yet passed, each round does mask_i |= mask_(j_i),
// j_i = j_(j_i), so a chain of n nodes takes ceil(log2 n) rounds.  A row read
// while its owner extends it only brings more true ancestors.  Depth = bits - 1.
// Latency bound (a few hundred bytes per sequence): what counts is the number
// of dependent steps, hence jumping and not a walk up from every node.
__global__ void __launch_bounds__(1024)
    tree_mask_kernel(const int32_t* parents, const int32_t* tree_lens, uint32_t* mask, int32_t* depth,
                     int T, int W, unsigned int* err) {
  extern __shared__ uint32_t sh[];
  uint32_t* m = sh;                                    // [T][W]
  int* jump = reinterpret_cast<int*>(sh + T * W);      // [T]
  const int b = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const int n = tree_lens != nullptr ? max(0, min(tree_lens[b], T)) : T;
  const int i = threadIdx.x;                           // node of this thread (blockDim >= T)
  for (int e = threadIdx.x; e < T * W; e += blockDim.x) {
    const int row = e / W, w = e - row * W;
    m[e] = row < n && row >> 5 == w ? 1u << (row & 31) : 0u;
  }
  if (i < T) {
    int j = -1;
    if (i < n) {
      j = parents[static_cast<int64_t>(b) * T + i];
      if (j < -1 || j >= i) {
        if (err) atomicOr(err, 1u << kErrTreeBadParent);
        j = -1;
      }
    }
    jump[i] = j;
  }
  __syncthreads();
  for (int round = 0; round < 10; ++round) {  // 2^10 >= T
    int more = 0;
    for (int e = threadIdx.x; e < T * W; e += blockDim.x) {
      const int row = e / W, j = jump[row];
      if (j >= 0) {
        m[e] |= m[j * W + (e - row * W)];
        more = 1;
      }
    }
    if (!__syncthreads_or(more)) break;
    const int j = i < T ? jump[i] : -1;
    const int nj = j >= 0 ? jump[j] : -1;
    __syncthreads();
    if (i < T) jump[i] = nj;
    __syncthreads();
  }
  uint32_t* out = mask + static_cast<int64_t>(b) * T * W;
  for (int e = threadIdx.x; e < T * W; e += blockDim.x) out[e] = m[e];
  if (i < T && depth != nullptr) {
    int d = -1;
    for (int w = 0; w < W; ++w) d += __popc(m[i * W + w]);
    depth[static_cast<int64_t>(b) * T + i] = max(d, 0);
  }
}

// Query tiles: qpt = 128 / g queries per 128-row tile, two tiles per unit when
// one does not hold all T nodes.
int queries_per_tile(int g) { return 128 / g; }

// Tile slots of the whole call, at most, and the end of a sequence's last tile:
// the kernels count both in 32 bits.
bool line_fits(int B, int units, int page_size, int max_pages) {
  if (static_cast<int64_t>(max_pages) * page_size > 0x7fffffffLL - 255) return false;
  return static_cast<double>(B) * units * ((static_cast<double>(max_pages) * page_size + 127) / 128 + 8) <
         2147483647.0;
}

// What the launches share: everything but the masks and the workspace.
attn_status tree_params(TreeParams* out, const void* q, const void* k_pool, const void* v_pool,
                        const int32_t* block_table, const int32_t* seqlens_k, void* o, float* lse, int B,
                        int T, int Hq, int Hkv, int d, bool bf16, int page_size, int num_pages, int max_pages,
                        const attn_opts* opts) {
  memset(out, 0, sizeof(*out));
  TreeParams& p = *out;
  int num_sms = 0;
  if (host_device_state(&p.err, &num_sms) != ATTN_OK) return ATTN_ERR_CUDA;
  const int g = Hq / Hkv;
  p.g = g;
  p.g_magic = (65536 + g - 1) / g;
  p.qpt = queries_per_tile(g);
  p.two_tiles = T > p.qpt ? 1 : 0;
  const int per = p.qpt * (p.two_tiles ? 2 : 1);
  p.units = Hkv * ((T + per - 1) / per);
  if (!line_fits(B, p.units, page_size, max_pages)) return ATTN_ERR_UNSUPPORTED;
  {
    const uint64_t eb = 2, row = static_cast<uint64_t>(d) * eb;
    const uint64_t dims[5] = {(uint64_t)d, (uint64_t)g, (uint64_t)Hkv, (uint64_t)T, (uint64_t)B};
    const uint64_t st[4] = {row, row * g, row * Hq, row * Hq * T};
    const uint32_t box[5] = {64, (uint32_t)g, 1, (uint32_t)p.qpt, 1};
    if (!host_make_map(&p.tm_q, q, bf16, 5, dims, st, box)) return ATTN_ERR_INVALID;
  }
  {
    const uint32_t box[3] = {64, 1, (uint32_t)(page_size < 128 ? page_size : 128)};
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)Hkv, (uint64_t)num_pages * page_size};
    const uint64_t st[2] = {(uint64_t)d * 2, (uint64_t)Hkv * d * 2};
    if (!host_make_map(&p.tm_k, k_pool, bf16, 3, dims, st, box)) return ATTN_ERR_INVALID;
    if (!host_make_map(&p.tm_v, v_pool, bf16, 3, dims, st, box)) return ATTN_ERR_INVALID;
  }
  p.block_table = block_table;
  p.seqlens_k = seqlens_k;
  p.o = o;
  p.lse = lse;
  p.sink = opts != nullptr ? opts->sink : nullptr;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.words = (T + 31) / 32;
  p.grid = num_sms < kTreeMaxCtas ? num_sms : kTreeMaxCtas;
  p.min_share = 4;
  p.unit_cost = 2;
  p.page_size = page_size;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.win_left = host_left(opts);
  p.sink_tokens = host_keep(opts);
  p.scale = host_scale(opts, d);
  p.scale_log2 = p.scale * kLog2e;
  p.softcap = opts != nullptr && opts->softcap > 0.0f ? opts->softcap : 0.0f;
  p.softcap_inv = p.softcap > 0.0f ? 1.0f / p.softcap : 0.0f;
  p.timeout_ns = host_timeout_ns();
  return ATTN_OK;
}

attn_status tree_launch(const TreeParams& p, int d, bool bf16, const char* what, cudaStream_t s) {
  const bool cap = p.softcap > 0.0f;
  char name[128];
  const int n = snprintf(name, sizeof(name), "attn_tree%s_paged_tcgen05_d%d_%s_%s_%s", what, d,
                         bf16 ? "bf16" : "f16", cap ? "softcap" : "nocap", p.two_tiles ? "m256" : "m128");
  if (p.o_part != nullptr) snprintf(name + n, sizeof(name) - n, "+attn_tree_merge_d%d", d);
  return host_finish(d == 64 ? launch_tree_d<64>(p, bf16, cap, s) : launch_tree_d<128>(p, bf16, cap, s), name);
}

}  // namespace

extern "C" {

attn_status attn_tree_mask(const int32_t* parents, const int32_t* tree_lens, uint32_t* mask,
                           int32_t* depth, int B, int T, void* stream) {
  if (B < 0 || T < 0) return ATTN_ERR_INVALID;
  if (T > ATTN_TREE_MAX_NODES) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return ATTN_OK;
  if (parents == nullptr || mask == nullptr || !host_aligned(parents, 4) || !host_aligned(mask, 4) ||
      !host_aligned(tree_lens, 4) || !host_aligned(depth, 4))
    return ATTN_ERR_INVALID;
  unsigned int* err = nullptr;
  if (host_device_state(&err, nullptr) != ATTN_OK) return ATTN_ERR_CUDA;
  const int W = (T + 31) / 32;
  constexpr int kMost = ATTN_TREE_MAX_NODES;
  int threads = (T * W + 31) / 32 * 32;
  if (threads > 1024) threads = 1024;
  const cudaError_t e = launch_pdl_upto<tree_mask_kernel>(
      (kMost * (kMost / 32) + kMost) * 4, dim3(B), threads, (T * W + T) * 4, static_cast<cudaStream_t>(stream), parents,
      tree_lens, mask, depth, T, W, err);
  return host_finish(e, "attn_tree_mask");
}

size_t attn_tree_workspace_bytes(int T, int Hq, int Hkv, int d) {
  if (T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > 128 || d <= 0) return 0;
  const size_t rows = T > queries_per_tile(Hq / Hkv) ? 256 : 128;
  return 2 * static_cast<size_t>(kTreeMaxCtas) * rows * (static_cast<size_t>(d) + 2) * sizeof(float) +
         kTreeMaxCtas * sizeof(int4);
}

attn_status attn_fwd_paged_tree(const void* q, const void* k_pool, const void* v_pool,
                                const int32_t* block_table, const int32_t* seqlens_k,
                                const uint32_t* tree_mask, const int32_t* tree_lens,
                                const int32_t* tree_depth, void* o, float* lse, int B, int T, int Hq,
                                int Hkv, int d, attn_dtype dtype, int page_size, int num_pages,
                                int max_pages_per_seq, void* workspace, size_t workspace_bytes,
                                const attn_opts* opts, void* stream) {
  if (B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || num_pages <= 0 || max_pages_per_seq <= 0)
    return ATTN_ERR_INVALID;
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return ATTN_ERR_UNSUPPORTED;
  const int g = Hq / Hkv;
  if (static_cast<int64_t>(num_pages) * page_size > 0x7fffffffLL ||
      !line_fits(1, 1, page_size, max_pages_per_seq) || T > ATTN_TREE_MAX_NODES || g > 128 || Hq > 65535)
    return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return ATTN_OK;
  if (q == nullptr || k_pool == nullptr || v_pool == nullptr || block_table == nullptr ||
      seqlens_k == nullptr || tree_mask == nullptr || o == nullptr)
    return ATTN_ERR_INVALID;
  for (const void* p : {q, k_pool, v_pool, static_cast<const void*>(o)})
    if (!host_aligned(p, 16)) return ATTN_ERR_INVALID;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seqlens_k),
                        static_cast<const void*>(tree_mask), static_cast<const void*>(tree_lens),
                        static_cast<const void*>(tree_depth), static_cast<const void*>(lse)})
    if (!host_aligned(p, 4)) return ATTN_ERR_INVALID;
  if (workspace == nullptr || !host_aligned(workspace, 16) ||
      workspace_bytes < attn_tree_workspace_bytes(T, Hq, Hkv, d))
    return ATTN_ERR_INVALID;
  const attn_status so = host_check_opts(opts, Hq, false);
  if (so != ATTN_OK) return so;
  // The mask says which nodes a row sees; only a left window applies beside it,
  // and it is measured from the node's depth.
  const bool window = opts != nullptr && opts->use_window;
  if (opts != nullptr && (opts->causal || opts->top_left || opts->alibi_slopes != nullptr ||
                          (window && opts->window_right >= 0)))
    return ATTN_ERR_UNSUPPORTED;
  const int left = window && opts->window_left >= 0 ? opts->window_left : -1;
  if (left >= 0 && tree_depth == nullptr) return ATTN_ERR_INVALID;

  TreeParams p;
  const attn_status st = tree_params(&p, q, k_pool, v_pool, block_table, seqlens_k, o, lse, B, T, Hq, Hkv, d,
                                     dtype == ATTN_BF16, page_size, num_pages, max_pages_per_seq, opts);
  if (st != ATTN_OK) return st;
  p.tree_lens = tree_lens;
  p.tree_mask = tree_mask;
  p.tree_depth = tree_depth;
  const size_t pieces = 2 * static_cast<size_t>(p.grid), rows = p.two_tiles ? 256 : 128;
  p.o_part = static_cast<float*>(workspace);
  p.ml_part = reinterpret_cast<float2*>(p.o_part + pieces * rows * d);
  p.cut = reinterpret_cast<int4*>(p.ml_part + pieces * rows);
  return tree_launch(p, d, dtype == ATTN_BF16, "", static_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace attn {

bool host_chain_applies(int B, int Lq, int Hq, int Hkv, int page_size, int max_pages, const attn_opts* opts) {
  const int g = Hq / Hkv;
  int sms = 0;
  if (opts == nullptr || host_device_state(nullptr, &sms) != ATTN_OK) return false;
  const int grid = sms < kTreeMaxCtas ? sms : kTreeMaxCtas;
  return host_keep(opts) > 0 && !opts->top_left &&
         opts->alibi_slopes == nullptr && (opts->causal || opts->window_right == 0 || Lq == 1) &&
         Lq <= queries_per_tile(g) && Hq <= 65535 && B <= 256 && static_cast<int64_t>(B) * Hkv >= 2 * grid &&
         line_fits(B, Hkv, page_size, max_pages);
}

attn_status host_chain(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
                       const int32_t* seqlens_k, void* o, float* lse, int B, int Lq, int Hq, int Hkv, int d,
                       bool bf16, int page_size, int num_pages, int max_pages, const attn_opts* opts,
                       cudaStream_t stream) {
  TreeParams p;
  const attn_status st = tree_params(&p, q, k_pool, v_pool, block_table, seqlens_k, o, lse, B, Lq, Hq, Hkv, d,
                                     bf16, page_size, num_pages, max_pages, opts);
  return st != ATTN_OK ? st : tree_launch(p, d, bf16, "_chain", stream);
}

}  // namespace attn
