// rope.cu -- rotary positions, and the write of new tokens' keys and values into
// a paged cache with the rotation on the way (attn_rope, attn_cache_append;
// include/attn_fwd.h states the rules).
//
// Pair i of a head turns by the angle position * f_i.  In 32 bits that angle is
// of little worth far out (at position 10^6 its rounding is 0.03 radians), so the
// kernels count in turns, in 64-bit fixed point: F_i = frac(f_i / 2 pi) * 2^64 as
// an integer, and position * F_i modulo 2^64 is the angle modulo a turn, exact
// but for F_i's own rounding (position * 2^-65 turns, and 2^-52 of f_i: 1 / 2 pi
// and the product).  Its upper half goes to sincospi, in 32 bits: cut to 2^-32 of
// a turn and rounded to 2^-25 of a half turn, 2^-23 radians together.
//
// Memory bound: every element is read and written once, about 4 operations each.
// A thread keeps the cosines and sines of its 8 pairs of one token and walks over
// heads with them, so that their cost (some 30 instructions a pair) is shared.  The
// work, (tile of tokens, head) in this order, is dealt to the CTAs that the GPU holds at
// once in equal runs: with a grid of tiles x groups of heads a third wave of a few
// CTAs ended the launch (2 x 8192 tokens of 32 + 8 heads: 66 us, so 55.3, where a copy of
// as many bytes takes 51.8).
#include "host.h"
#include "launch.h"
#include "overlap.h"
#include "ptx.cuh"

#include <algorithm>
#include <cmath>

using namespace attn;

namespace {

constexpr int kThreads = 256;
// CTAs that an SM holds.  At 3, 4, 5 and 6: 57.1, 54.8, 62.2 and 68.3 us for that prompt, in fp16
// by pairs 57.4, 54.8, 60.4 and 75.5, of 32 heads of d = 64 25.7, 24.6, 27.5 and 31.6; 2000 tokens
// of those 6.0, 7.3, 7.9 and 10.9, 300 tokens of 10 heads 3.2 to 3.7; 4096 tokens into the
// cache 22.2, 20.9, 22.0 and 25.1.
constexpr int kPerSm = 4;
constexpr int kMaxDim = 512;

// A tensor's rows: element strides of batch, head and row.
struct Rows {
  const void* src;
  void* dst;
  attn_strides in, out;
  int heads;
};

struct RopeParams {
  Rows part[3];  // q, k, v; a part of the cache goes to row slots[token] (out.row, out.head used)
  const int32_t* positions;
  int64_t pos_batch;
  const int32_t* slots;  // nullptr: part[1] is written like part[0]
  int64_t num_slots;
  const double* inv_freq;
  int tokens, L, d, rot;  // tokens = batch * L
  int share, extra;       // entries of the (tile, head) list per CTA, and CTAs with one more
  int interleaved;
  float sign, scale;      // sign -1: the inverse rotation
  unsigned int* err;
};

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return __half22float2(h);
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
  return BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}

// 2^64 times the fraction of a turn per position.
__device__ __forceinline__ unsigned long long turns_of(double f) {
  double t = f * 0.15915494309189535;  // 1 / 2 pi
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // (a fraction that rounds to 1 saturates: 2^-64 off)
}

// Cosine and sine of the angle at `pos`, times the rotation's scale.
__device__ __forceinline__ void turn(unsigned long long f, int pos, float sign, float scale, float& c, float& s) {
  const unsigned long long a = f * static_cast<unsigned long long>(static_cast<long long>(pos));
  const float half_turns = static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half_turns, &s, &c);
  s *= sign * scale;
  c *= scale;
}

// Where head `h` of the call (q's heads, then k's, then v's) of a token is read
// and written; false: not written (padding, or a slot out of range).
struct Place {
  const uint4* src;
  uint4* dst;
  bool rotate, write;
};
__device__ __forceinline__ Place place(const RopeParams& p, int h, int b, int l, int64_t slot) {
  int i = 0;
  if (h >= p.part[0].heads) {
    h -= p.part[0].heads;
    i = 1;
    if (h >= p.part[1].heads) {
      h -= p.part[1].heads;
      i = 2;
    }
  }
  const Rows& r = p.part[i];
  const uint16_t* src = static_cast<const uint16_t*>(r.src) + b * r.in.batch + h * r.in.head + l * r.in.row;
  uint16_t* dst = static_cast<uint16_t*>(r.dst) + h * r.out.head;
  bool write = true;
  if (i > 0 && p.slots != nullptr) {
    write = slot >= 0;
    dst += slot * r.out.row;
  } else {
    dst += b * r.out.batch + l * r.out.row;
  }
  return {reinterpret_cast<const uint4*>(src), reinterpret_cast<uint4*>(dst), i < 2, write};
}

// The token's slot, or -1 where its rows are not written.
__device__ __forceinline__ int64_t slot_of(const RopeParams& p, int token) {
  if (p.slots == nullptr) return -1;
  const int s = p.slots[token];
  if (s >= 0 && s < p.num_slots) return s;
  if (s != -1 && p.err) atomicOr(p.err, 1u << kErrCacheBadIndex);
  return -1;
}

// This CTA's run of the (tile, head) list: the tile, and heads [h0, h1) of it, then
// the next tile's.  (A tile has as many tokens as the CTA has rows of threads.)
struct Run {
  int left, tile, h0;
  __device__ __forceinline__ Run(const RopeParams& p, int heads) {
    const int cta = blockIdx.x, first = cta * p.share + min(cta, p.extra);
    left = p.share + (cta < p.extra ? 1 : 0);
    tile = first / heads;
    h0 = first - tile * heads;
  }
  __device__ __forceinline__ int end(int heads) const { return min(heads, h0 + left); }
  __device__ __forceinline__ void next(int h1) {
    left -= h1 - h0;
    h0 = 0;
    ++tile;
  }
};

// Rows of which both halves of every pair lie in whole 16-byte pieces (rot a
// multiple of 16): a thread owns two pieces, 8 pairs, or one piece behind the
// rotated elements.  Neighbouring threads take neighbouring pieces of a row, then
// the next token's.
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, kPerSm) rope_pairs_kernel(const RopeParams p) {
  __shared__ unsigned long long freq[kMaxDim / 2];
  pdl_launch_dependents();
  pdl_wait();
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) freq[i] = turns_of(p.inv_freq[i]);
  __syncthreads();
  const int turned = p.rot / 16, units = turned + (p.d - p.rot) / 8;
  const int per = kThreads / units;  // tokens of a tile
  const int tt = threadIdx.x / units, u = threadIdx.x - tt * units;
  const bool rot = u < turned;
  // First and second piece of the thread, in pieces of 8 elements.
  const int e0 = rot ? (INTER ? 2 * u : u) : 2 * turned + (u - turned);
  const int e1 = rot ? (INTER ? 2 * u + 1 : turned + u) : e0;
  const int heads = p.part[0].heads + p.part[1].heads + p.part[2].heads;
  for (Run run(p, heads); run.left > 0;) {
    const int h0 = run.h0, h1 = run.end(heads), token = run.tile * per + tt;
    run.next(h1);
    if (tt >= per || token >= p.tokens) continue;
    const int b = token / p.L, l = token - b * p.L;
    const int64_t slot = slot_of(p, token);
    float c[8], s[8];
    if (rot) {
      const int pos = p.positions != nullptr ? p.positions[b * p.pos_batch + l] : l;
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(freq[8 * u + i], pos, p.sign, p.scale, c[i], s[i]);
    }
    // The next head's pieces are on their way while this one's are turned.
    Place now = place(p, h0, b, l, slot);
    uint4 x = now.src[e0], y = now.src[e1];
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
      Place next = now;
      uint4 nx = x, ny = y;
      if (h + 1 < h1) {
        next = place(p, h + 1, b, l, slot);
        nx = next.src[e0];
        ny = next.src[e1];
      }
      if (now.write) {
        if (rot && now.rotate) {
          const uint32_t a[4] = {x.x, x.y, x.z, x.w}, d[4] = {y.x, y.y, y.z, y.w};
          uint32_t oa[4], od[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 fa = widen<BF16>(a[i]), fd = widen<BF16>(d[i]);
            if constexpr (INTER) {  // a: pairs i, d: pairs 4 + i
              oa[i] = narrow<BF16>(fa.x * c[i] - fa.y * s[i], fa.y * c[i] + fa.x * s[i]);
              od[i] = narrow<BF16>(fd.x * c[4 + i] - fd.y * s[4 + i], fd.y * c[4 + i] + fd.x * s[4 + i]);
            } else {
              oa[i] = narrow<BF16>(fa.x * c[2 * i] - fd.x * s[2 * i], fa.y * c[2 * i + 1] - fd.y * s[2 * i + 1]);
              od[i] = narrow<BF16>(fd.x * c[2 * i] + fa.x * s[2 * i], fd.y * c[2 * i + 1] + fa.y * s[2 * i + 1]);
            }
          }
          x = make_uint4(oa[0], oa[1], oa[2], oa[3]);
          y = make_uint4(od[0], od[1], od[2], od[3]);
        }
        now.dst[e0] = x;
        if (rot) now.dst[e1] = y;
      }
      now = next;
      x = nx;
      y = ny;
    }
  }
}

// Any even rot: a thread owns one piece of 8 elements and finds their partners in
// shared memory, where the CTA has put its rows of the head before any of them is
// written (the output may be the input).  126 of 128 elements, 2 x 8192 tokens of 40
// heads: 82.8 us where the form above takes 55.3.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, kPerSm) rope_any_kernel(const RopeParams p) {
  __shared__ unsigned long long freq[kMaxDim / 2];
  __shared__ uint4 rows[2][kThreads];
  pdl_launch_dependents();
  pdl_wait();
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) freq[i] = turns_of(p.inv_freq[i]);
  __syncthreads();
  const int units = p.d / 8, per = kThreads / units;
  const int tt = threadIdx.x / units, u = threadIdx.x - tt * units;
  const int heads = p.part[0].heads + p.part[1].heads + p.part[2].heads;
  int buf = 0;
  for (Run run(p, heads); run.left > 0;) {
    const int h0 = run.h0, h1 = run.end(heads), token = run.tile * per + tt;
    run.next(h1);
    const bool mine = tt < per && token < p.tokens;
    const int b = mine ? token / p.L : 0, l = mine ? token - b * p.L : 0;
    const int pos = !mine ? 0 : p.positions != nullptr ? p.positions[b * p.pos_batch + l] : l;
    const int64_t slot = mine ? slot_of(p, token) : -1;
    // The partner of each element, and out = x c + partner s.
    float c[8], s[8];
    int at[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 8 * u + i, half = p.rot / 2;
      at[i] = -1;
      c[i] = 1.0f;
      s[i] = 0.0f;
      if (e < p.rot) {
        const bool second = p.interleaved ? (e & 1) : e >= half;
        const int pair = p.interleaved ? e >> 1 : second ? e - half : e;
        at[i] = p.interleaved ? (e ^ 1) : second ? e - half : e + half;
        turn(freq[pair], pos, p.sign, p.scale, c[i], s[i]);
        if (!second) s[i] = -s[i];
      }
    }
    // The next head's pieces are on their way while this one's are turned.
    Place w{nullptr, nullptr, false, false};
    uint4 nx = make_uint4(0, 0, 0, 0);
    if (mine) nx = place(p, h0, b, l, slot).src[u];
    for (int h = h0; h < h1; ++h, buf ^= 1) {
      uint4 x = nx;
      if (mine) {
        w = place(p, h, b, l, slot);
        if (h + 1 < h1) nx = place(p, h + 1, b, l, slot).src[u];
      }
      rows[buf][threadIdx.x] = x;
      __syncthreads();  // (one a round: the buffer written next was read before this one)
      if (!w.write) continue;
      if (w.rotate) {
        const uint16_t* row = reinterpret_cast<const uint16_t*>(&rows[buf][tt * units]);
        uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (at[2 * i] < 0) continue;  // (elements behind the rotated ones keep their bits; rot is even)
          const float2 f = widen<BF16>(v[i]);
          const float2 g = widen<BF16>(row[at[2 * i]] | (static_cast<uint32_t>(row[at[2 * i + 1]]) << 16));
          v[i] = narrow<BF16>(f.x * c[2 * i] + g.x * s[2 * i], f.y * c[2 * i + 1] + g.y * s[2 * i + 1]);
        }
        x = make_uint4(v[0], v[1], v[2], v[3]);
      }
      w.dst[u] = x;
    }
  }
}

bool strides_ok(const attn_strides& s, bool batch) {
  return s.head > 0 && s.row > 0 && s.head % 8 == 0 && s.row % 8 == 0 && (!batch || (s.batch > 0 && s.batch % 8 == 0));
}

// What the options ask for; ATTN_OK and rot = 0 without them.
attn_status read_rope(const attn_rope_opts* r, int d, RopeParams& p) {
  p.sign = 1.0f;
  p.scale = 1.0f;
  if (r == nullptr) return ATTN_OK;
  if (r->rotary_dim < 0 || r->rotary_dim > d || r->rotary_dim % 2 != 0) return ATTN_ERR_INVALID;
  if (r->rotary_dim > 0 && (r->inv_freq == nullptr || !host_aligned(r->inv_freq, 8))) return ATTN_ERR_INVALID;
  if (!(r->scale >= 0.0f) || std::isinf(r->scale)) return ATTN_ERR_INVALID;
  p.inv_freq = r->inv_freq;
  p.rot = r->rotary_dim;
  p.interleaved = r->interleaved ? 1 : 0;
  p.sign = r->inverse ? -1.0f : 1.0f;
  p.scale = r->scale > 0.0f ? r->scale : 1.0f;
  return ATTN_OK;
}

attn_status launch(RopeParams& p, bool bf16, cudaStream_t stream, const char* name) {
  int sms = 0;
  if (host_device_state(&p.err, &sms) != ATTN_OK) return ATTN_ERR_CUDA;
  const bool pairs = p.rot % 16 == 0;
  const int units = pairs ? p.rot / 16 + (p.d - p.rot) / 8 : p.d / 8;
  const int per = kThreads / units;
  const int heads = p.part[0].heads + p.part[1].heads + p.part[2].heads;
  const int64_t work = (static_cast<int64_t>(p.tokens) + per - 1) / per * heads;
  if (work > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;  // (more than the GPU's memory holds)
  const int grid = static_cast<int>(std::min<int64_t>(work, static_cast<int64_t>(kPerSm) * sms));
  p.share = static_cast<int>(work / grid);
  p.extra = static_cast<int>(work % grid);
  cudaError_t e;
  if (pairs && p.interleaved)
    e = bf16 ? launch_pdl(rope_pairs_kernel<true, true>, grid, kThreads, 0, stream, p)
             : launch_pdl(rope_pairs_kernel<false, true>, grid, kThreads, 0, stream, p);
  else if (pairs)
    e = bf16 ? launch_pdl(rope_pairs_kernel<true, false>, grid, kThreads, 0, stream, p)
             : launch_pdl(rope_pairs_kernel<false, false>, grid, kThreads, 0, stream, p);
  else
    e = bf16 ? launch_pdl(rope_any_kernel<true>, grid, kThreads, 0, stream, p)
             : launch_pdl(rope_any_kernel<false>, grid, kThreads, 0, stream, p);
  return host_finish(e, name);
}

// Whether a part's output shares memory with an input that other threads read: an input of other
// rows, or its own other than in place.
bool over_inputs(const RopeParams& p, int inputs) {
  const int B = p.tokens / p.L;
  const auto in = [&](int i) { return Extent{p.part[i].src, p.part[i].in, {B, p.part[i].heads, p.L}, p.d}; };
  for (int i = 0; i < (p.slots != nullptr ? 1 : 2); ++i) {
    if (p.part[i].heads == 0) continue;
    const Extent out{p.part[i].dst, p.part[i].out, {B, p.part[i].heads, p.L}, p.d};
    for (int j = 0; j < inputs; ++j)
      if (p.part[j].heads > 0 && !(i == j && same_rows(out, in(j))) && overlap(out, in(j))) return true;
    const Extent other{p.part[1].dst, p.part[1].out, {B, p.part[1].heads, p.L}, p.d};
    if (i == 0 && p.slots == nullptr && p.part[1].heads > 0 && overlap(out, other)) return true;
  }
  return false;
}

attn_status check_dim(int d) {
  if (d <= 0) return ATTN_ERR_INVALID;
  return d % 8 != 0 || d > kMaxDim ? ATTN_ERR_UNSUPPORTED : ATTN_OK;
}

}  // namespace

extern "C" {

attn_status attn_rope_freqs(int rotary_dim, double base, attn_rope_scaling scaling, double factor,
                            double original_len, double slow_turns, double fast_turns, double* inv_freq) {
  if (rotary_dim <= 0 || rotary_dim % 2 != 0 || inv_freq == nullptr || !(base > 1.0) || std::isinf(base))
    return ATTN_ERR_INVALID;
  if (scaling < ATTN_ROPE_PLAIN || scaling > ATTN_ROPE_RAMP) return ATTN_ERR_INVALID;
  if (scaling != ATTN_ROPE_PLAIN && (!(factor >= 1.0) || std::isinf(factor))) return ATTN_ERR_INVALID;
  const bool parts = scaling == ATTN_ROPE_PARTS || scaling == ATTN_ROPE_RAMP;
  if (parts && (!(original_len > 0.0) || std::isinf(original_len) || !(slow_turns > 0.0) ||
                !(fast_turns > slow_turns) || std::isinf(fast_turns)))
    return ATTN_ERR_INVALID;
  constexpr double kTwoPi = 6.283185307179586;
  const double r = rotary_dim;
  if (scaling == ATTN_ROPE_BASE) {
    if (rotary_dim <= 2) return ATTN_ERR_INVALID;
    base *= std::pow(factor, r / (r - 2.0));
  }
  // The index at which a pair makes `turns` turns in original_len positions.
  auto index_of = [&](double turns) { return r * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(base)); };
  double low = 0.0, high = 0.0;
  if (scaling == ATTN_ROPE_RAMP) {
    low = std::max(0.0, std::floor(index_of(fast_turns)));
    high = std::min(r - 1.0, std::ceil(index_of(slow_turns)));
    if (high <= low) high = low + 0.001;
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (scaling == ATTN_ROPE_LINEAR) f /= factor;
    if (parts) {
      double keep;  // 1: as it is, 0: slowed by the factor
      if (scaling == ATTN_ROPE_PARTS)
        keep = (original_len * f / kTwoPi - slow_turns) / (fast_turns - slow_turns);
      else
        keep = 1.0 - (i - low) / (high - low);
      keep = std::min(1.0, std::max(0.0, keep));
      f = f * keep + f / factor * (1.0 - keep);
    }
    inv_freq[i] = f;
  }
  return ATTN_OK;
}

attn_status attn_rope(const void* q, void* q_out, const void* k, void* k_out, const int32_t* positions,
                      int64_t positions_batch_stride, int B, int L, int Hq, int Hkv, int d, attn_dtype dtype,
                      attn_strides sq, attn_strides sq_out, attn_strides sk, attn_strides sk_out,
                      const attn_rope_opts* rope, void* stream) {
  if (B < 0 || L < 0 || Hq < 0 || Hkv < 0 || rope == nullptr || positions_batch_stride < 0) return ATTN_ERR_INVALID;
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return dtype == ATTN_E4M3 ? ATTN_ERR_UNSUPPORTED : ATTN_ERR_INVALID;
  const attn_status dim = check_dim(d);
  if (dim != ATTN_OK) return dim;
  RopeParams p{};
  const attn_status st = read_rope(rope, d, p);
  if (st != ATTN_OK) return st;
  if (static_cast<int64_t>(B) * L > 0x7fffffffLL - 256) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || L == 0 || Hq + static_cast<int64_t>(Hkv) == 0) return ATTN_OK;
  if (Hq + static_cast<int64_t>(Hkv) > 65535) return ATTN_ERR_UNSUPPORTED;
  if (!host_aligned(positions, 4)) return ATTN_ERR_INVALID;
  if (Hq > 0 && (q == nullptr || q_out == nullptr || !host_aligned(q, 16) || !host_aligned(q_out, 16) ||
                 !strides_ok(sq, B > 1) || !strides_ok(sq_out, B > 1)))
    return ATTN_ERR_INVALID;
  if (Hkv > 0 && (k == nullptr || k_out == nullptr || !host_aligned(k, 16) || !host_aligned(k_out, 16) ||
                  !strides_ok(sk, B > 1) || !strides_ok(sk_out, B > 1)))
    return ATTN_ERR_INVALID;
  p.part[0] = Rows{q, q_out, sq, sq_out, Hq};
  p.part[1] = Rows{k, k_out, sk, sk_out, Hkv};
  p.positions = positions;
  p.pos_batch = positions_batch_stride;
  p.tokens = B * L;
  p.L = L;
  p.d = d;
  if (over_inputs(p, 2)) return ATTN_ERR_INVALID;
  return launch(p, dtype == ATTN_BF16, static_cast<cudaStream_t>(stream), "attn_rope");
}

attn_status attn_cache_append(const void* q, void* q_out, const void* k, const void* v, void* k_pool, void* v_pool,
                              const int32_t* slots, const int32_t* positions, int num_tokens, int Hq, int Hkv, int d,
                              attn_dtype dtype, int page_size, int num_pages, attn_strides sq, attn_strides sq_out,
                              attn_strides sk, attn_strides sv, const attn_rope_opts* rope, void* stream) {
  if (num_tokens < 0 || Hq < 0 || Hkv <= 0 || page_size <= 0 || num_pages <= 0) return ATTN_ERR_INVALID;
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return dtype == ATTN_E4M3 ? ATTN_ERR_UNSUPPORTED : ATTN_ERR_INVALID;
  const attn_status dim = check_dim(d);
  if (dim != ATTN_OK) return dim;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return ATTN_ERR_UNSUPPORTED;
  RopeParams p{};
  const attn_status st = read_rope(rope, d, p);
  if (st != ATTN_OK) return st;
  if (rope != nullptr && rope->inverse) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_pages) * page_size > 0x7fffffffLL || num_tokens > 0x7fffffff - 256 ||
      Hq + 2 * static_cast<int64_t>(Hkv) > 65535)
    return ATTN_ERR_UNSUPPORTED;
  if (num_tokens == 0) return ATTN_OK;
  if (slots == nullptr || !host_aligned(slots, 4) || !host_aligned(positions, 4) || (p.rot > 0 && positions == nullptr))
    return ATTN_ERR_INVALID;
  for (const void* x : {k, v, static_cast<const void*>(k_pool), static_cast<const void*>(v_pool)})
    if (x == nullptr || !host_aligned(x, 16)) return ATTN_ERR_INVALID;
  if (!strides_ok(sk, false) || !strides_ok(sv, false)) return ATTN_ERR_INVALID;
  if (Hq > 0 && (q == nullptr || q_out == nullptr || !host_aligned(q, 16) || !host_aligned(q_out, 16) ||
                 !strides_ok(sq, false) || !strides_ok(sq_out, false)))
    return ATTN_ERR_INVALID;
  const attn_strides pool{0, d, static_cast<int64_t>(Hkv) * d};
  p.part[0] = Rows{q, q_out, sq, sq_out, Hq};
  p.part[1] = Rows{k, k_pool, sk, pool, Hkv};
  p.part[2] = Rows{v, v_pool, sv, pool, Hkv};
  p.positions = positions;
  p.slots = slots;
  p.num_slots = static_cast<int64_t>(num_pages) * page_size;
  p.tokens = num_tokens;
  p.L = num_tokens;
  p.d = d;
  if (over_inputs(p, 3)) return ATTN_ERR_INVALID;
  return launch(p, dtype == ATTN_BF16, static_cast<cudaStream_t>(stream), "attn_cache_append");
}

}  // extern "C"
