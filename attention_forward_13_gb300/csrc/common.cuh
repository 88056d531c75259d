// common.cuh -- parameter blocks and small device helpers shared by the
// attention kernels of this library (prefill, paged decode, combine).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

// Bytes of each output row the dense prefill epilogue stages and stores per
// round (one TMA store per softmax warp and round): 128 without PackGQA, 64
// with packed heads (measured) and for FP8 (whose widened V buffers take the
// shared memory a 128-byte stage would need).
#ifndef ATTN_O_ROUND_BYTES
#define ATTN_O_ROUND_BYTES 128
#endif

namespace attn {

constexpr int prefill_o_round_bytes(bool fp8, int pack) {
  return (fp8 || pack > 1) ? 64 : ATTN_O_ROUND_BYTES;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Device error word bits (one per wait site / check).
enum ErrBits : uint32_t {
  kErrPrefillQ = 0,
  kErrPrefillKFull = 1,
  kErrPrefillVFull = 2,
  kErrPrefillKEmpty = 3,
  kErrPrefillVEmpty = 4,
  kErrPrefillSFull = 5,
  kErrPrefillPFull = 6,
  kErrPrefillOFinal = 7,
  kErrPrefillTeardown = 8,
  kErrPrefillBadPage = 9,
  kErrDecodeFull = 12,
  kErrDecodeEmpty = 13,
  kErrDecodeBadPage = 14,
  kErrDecodeTeardown = 15,
  kErrSelftest = 20,
  kErrTreeWait = 21,
  kErrTreeBadPage = 22,
  kErrTreeTeardown = 23,
  kErrTreeBadParent = 24,
  kErrCacheBadIndex = 25,
  kErrLinearWait = 26,
  kErrLinearTeardown = 27,
};

// Element types of a prefill instantiation: fp16 / bf16 end to end, or e4m3
// Q/K/V/O (FP8 static quantisation: S on the kind::f8f6f4 tensor path, V
// widened to fp16 on chip for P.V, O scaled and saturated to e4m3).
enum PrefillDt : int { kDtF16 = 0, kDtBF16 = 1, kDtE4M3 = 2 };

// Mask of a prefill instantiation: none, the causal / window band, or the band
// with the first sink_tokens keys visible left of it.
enum PrefillMask : int { kMaskNone = 0, kMaskBand = 1, kMaskBandKeep = 2 };

// Score transform of a prefill instantiation (applied to the raw score
// before masking).
enum ScoreXf : int { kXfNone = 0, kXfSoftcap = 1, kXfAlibi = 2, kXfBias = 3 };

// Bounds of the host-packed static schedule carried in PrefillParams, chosen
// so that the launch parameters stay within 4 KB.
constexpr int kSchedMaxCtas = 160;
constexpr int kSchedMaxItems = 1408;

// Prefill (dense / varlen) launch parameters.  Tensor maps are 4-D
// (d, rows, heads, batch); varlen problems use one batch slot and a row base.
struct PrefillParams {
  CUtensorMap tm_q;
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  // Dense problems whose softmax warps each own 32 consecutive queries of one
  // head (no packing, or at most 4 heads per tile): the epilogue stores O and
  // LSE by TMA through these maps (o_tma / lse_tma nonzero).  O: 4-D
  // (d, Lq, Hq, B), box {o_tma bytes of d (64 or 128), 32 rows, 1, 1},
  // swizzle of the same width; LSE: 3-D (Lq, Hq, B) fp32, box {32, 1, 1}.
  // Rows past Lq fall outside the maps and are not written.
  CUtensorMap tm_o;
  CUtensorMap tm_lse;
  int o_tma, lse_tma;  // o_tma: bytes of each row per store (0: no map)
  void* o;
  float* lse;
  int64_t o_row, o_head, o_batch;  // element strides of O
  int64_t lse_head, lse_batch;     // element strides of LSE (row stride 1)
  const int32_t* cu_q;             // varlen: [B+1] (nullptr in batch mode)
  const int32_t* cu_k;
  const float* sink;               // [Hq] or nullptr
  int B, Hq, Hkv, Lq, Lk;          // batch-mode lengths (ignored for varlen)
  int total_q, total_k;            // varlen: packed extents (sequences are clamped to them)
  // Query heads per work item (PackGQA): 1, or g = Hq / Hkv when the g query
  // heads of a kv head share every tile.  A 128-row tile then holds
  // qpt = 128 / pack queries of each of the pack heads, head-major (row
  // r <-> head h0 + (r >> qpt_log2), query m0 + (r & (qpt - 1))), as one
  // TMA box {d, qpt queries, pack heads} lands them.
  int pack;
  int qpt_log2;                    // log2(queries per 128-row tile)
  int units;                       // Hq / pack: head groups per batch
  int num_m_blocks;                // query blocks (two tiles) per (b, head group)
  int num_items;                   // num_m_blocks * B * units work items
  float scale_log2;                // scale * log2(e)
  float scale;                     // plain scale (soft-cap path)
  float softcap;                   // cap (> 0 when the soft-cap variant runs)
  float softcap_inv;               // 1 / cap
  // Key bounds of query row i (bottom-right aligned): i + Lk - Lq - win_left
  // <= j <= i + Lk - Lq + win_right; a negative bound is unbounded.  Causal
  // masking is win_right = 0.  Only read by the masked instantiations.
  int win_left, win_right;
  int sink_tokens;                 // keys j < sink_tokens stay visible left of the band (win_left >= 0)
  int fold;                        // > 0: first tokens share the band's first tile (see below)
  int top_left;                    // masks and ALiBi aligned top-left (row i on key i)
  float o_scale;                   // FP8 static quantisation: scale_p * scale_o on O
  float inv_scale;                 // 1 / scale (bias and ALiBi go to raw-score units)
  const float* alibi;              // ALiBi slopes, (b, h) at b * alibi_stride + h
  int alibi_stride;
  const void* bias;                // elementwise bias (input dtype), batch mode only
  int64_t bias_row, bias_head, bias_batch;  // its element strides (key stride 1)
  // Paged KV cache (chunked prefill): tm_k / tm_v are then 3-D maps
  // (d, Hkv, num_pages * page_size) over the pools, and sequence b has
  // seqlens_k[b] keys; nullptr otherwise.
  const int32_t* block_table;
  const int32_t* seqlens_k;
  int page_size, max_pages, num_pages;
  unsigned int* err;
  uint64_t timeout_ns;
  // Dense masked problems: a static assignment of the work items to CTAs,
  // packed on the host (sched_n > 0).  CTA c takes items
  // sched_item[sched_off[c]] .. sched_item[sched_off[c + 1] - 1] in order;
  // sched_n == 0: the snake order over the plain item list.
  int sched_n;
  uint16_t sched_off[kSchedMaxCtas + 1];
  uint16_t sched_item[kSchedMaxItems];
};
static_assert(sizeof(PrefillParams) <= 4096, "prefill launch parameters exceed 4 KB");

// Launch parameters of the windows whose first tokens stay visible.  With
// fold > 0 (sink_tokens rounded up to 8, at most 64; dense and group mode) the
// tiles of an item start at fold keys before its band, and rows 0 .. fold - 1
// of its first tile are keys 0 .. fold - 1 in place of those: one box of fold
// rows and one of 128 - fold.  (Eight rows are one swizzle period.)
struct PrefillKeepParams : PrefillParams {
  CUtensorMap tm_k_first, tm_k_rest, tm_v_first, tm_v_rest;
};

// Paged split-KV decode parameters.
struct DecodeParams {
  CUtensorMap tm_k;  // 3-D (d, Hkv, num_pages * page_size)
  CUtensorMap tm_v;
  const void* q;     // [B][Lq][Hq][d]
  const int32_t* block_table;
  const int32_t* seqlens_k;
  void* o;           // final O [B][Lq][Hq][d] (num_splits == 1)
  float* lse;        // final LSE [B][Hq][Lq] or nullptr (num_splits == 1)
  float* o_part;     // [S][B][Hq][Lq][d] (num_splits > 1)
  float* lse_part;   // [S][B][Hq][Lq]
  const float* sink; // [Hq] or nullptr (used only when num_splits == 1)
  int B, Lq, Hq, Hkv, page_size, num_pages, max_pages, num_splits, chunk_pages;
  float scale_log2, scale, softcap, softcap_inv;
  int win_left, win_right;  // as in PrefillParams (causal is win_right = 0)
  int sink_tokens;
  int top_left;
  const float* alibi;       // ALiBi slopes as in PrefillParams, or nullptr
  int alibi_stride;
  unsigned int* err;
  uint64_t timeout_ns;
};

// Tree attention over a paged cache (tree_kernel.cuh).
constexpr int kTreeMaxCtas = 160;  // bounds the workspace; more SMs than that stay idle
struct TreeParams {
  CUtensorMap tm_q;  // 5-D (d, g, Hkv, T, B), box {64, g, 1, qpt, 1}
  CUtensorMap tm_k;  // 3-D (d, Hkv, num_pages * page_size)
  CUtensorMap tm_v;
  const int32_t* block_table;
  const int32_t* seqlens_k;
  const int32_t* tree_lens;   // nodes per sequence, or nullptr: T each
  const uint32_t* tree_mask;  // [B][T][words]
  const int32_t* tree_depth;  // [B][T], or nullptr: 0
  void* o;                    // [B][T][Hq][d]
  float* lse;                 // [B][Hq][T] or nullptr
  const float* sink;          // [Hq] or nullptr
  float* o_part;              // [2 * grid][d / 4][rows][4], rows = 128 or 256
  float2* ml_part;            // [2 * grid][rows]
  int4* cut;                  // [grid] for the merge kernel: the unit to merge there
  int B, T, Hq, Hkv, g, words;
  int g_magic;                // ceil(2^16 / g)
  int qpt;                    // queries per 128-row tile
  int two_tiles;              // units of two query tiles
  int units;                  // (query block, kv head) pairs per sequence
  int grid, min_share;        // CTAs, and the fewest slots worth a CTA
  int unit_cost;              // slots of the line that a unit takes beside its tiles (>= 1)
  int page_size, page_log2, num_pages, max_pages;
  int win_left, sink_tokens;
  float scale_log2, scale, softcap, softcap_inv;
  unsigned int* err;
  uint64_t timeout_ns;
};

struct CombineParams {
  const float* o_part;
  const float* lse_part;
  const float* sink;
  void* o;
  float* lse;
  int num_splits, B, Hq, Lq, d;
};

}  // namespace attn
