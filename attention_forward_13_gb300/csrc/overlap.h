// overlap.h -- whether two strided tensors share memory (host only).  The kernels that write
// one while other CTAs read the other refuse such calls: what they gave would depend on
// which CTA came first.
#pragma once
#include "../../include/attn_fwd.h"

#include <algorithm>
#include <cstdint>

namespace attn {

// Rows of `width` neighbouring 16-bit elements: batch, head and row.
struct Extent {
  const void* base;
  attn_strides s;  // elements
  int64_t n[3];    // of batches, heads, rows
  int64_t width;

  int64_t stride(int i) const { return i == 0 ? s.batch : i == 1 ? s.head : s.row; }
  int64_t span() const {  // elements from the first to behind the last
    int64_t x = width;
    for (int i = 0; i < 3; ++i) x += (n[i] - 1) * (n[i] > 1 ? stride(i) : 0);
    return x;
  }
};

inline bool same_rows(const Extent& a, const Extent& b) {
  for (int i = 0; i < 3; ++i)
    if (a.n[i] > 1 && a.stride(i) != b.stride(i)) return false;
  return a.base == b.base;
}

// Two rows share an element when the distance between their starts is below the width.  The
// distances are `at` plus a sum of strides times counts: one side's counts up, the other's
// down, equal strides taken together.
class RowSearch {
 public:
  RowSearch(const Extent& a, const Extent& b) : width_(a.width) {
    for (int i = 0; i < 3; ++i) {
      add(a, i, -(a.n[i] - 1), 0);
      add(b, i, 0, b.n[i] - 1);
    }
    std::sort(t_, t_ + terms_, [](const Term& x, const Term& y) { return x.stride > y.stride; });
  }
  // From the largest stride down, only over counts from which the rest can still reach 0: a
  // few for each stride of tensors whose dimensions nest.  Others might take long; after
  // a few thousand steps the answer is no, as it is for all that nothing is known of.
  bool find(int64_t at, int k = 0) {
    if (k == terms_) return at > -width_ && at < width_;
    if (++steps_ > 4096) return false;
    int64_t lo = 0, hi = 0;
    for (int i = k + 1; i < terms_; ++i) {
      lo += t_[i].lo * t_[i].stride;
      hi += t_[i].hi * t_[i].stride;
    }
    const int64_t s = t_[k].stride;
    const int64_t first = std::max(t_[k].lo, -floor_div(at + hi + width_ - 1, s));
    const int64_t last = std::min(t_[k].hi, floor_div(width_ - 1 - at - lo, s));
    for (int64_t c = first; c <= last && steps_ <= 4096; ++c)
      if (find(at + c * s, k + 1)) return true;
    return false;
  }

 private:
  struct Term {
    int64_t stride, lo, hi;
  };
  static int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && a < 0 ? 1 : 0); }
  void add(const Extent& e, int i, int64_t lo, int64_t hi) {
    if (e.n[i] <= 1) return;
    for (int j = 0; j < terms_; ++j)
      if (t_[j].stride == e.stride(i)) {
        t_[j].lo += lo;
        t_[j].hi += hi;
        return;
      }
    t_[terms_++] = Term{e.stride(i), lo, hi};
  }
  Term t_[6];
  int terms_ = 0, steps_ = 0;
  int64_t width_;
};

// Both of the same width and of positive strides, at addresses that are multiples of 2 bytes.
inline bool overlap(const Extent& a, const Extent& b) {
  const int64_t at = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.base)) -
                      static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.base))) / 2;
  if (at >= a.span() || -at >= b.span()) return false;
  return RowSearch(a, b).find(at);
}

}  // namespace attn
