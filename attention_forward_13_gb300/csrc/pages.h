// pages.h -- how many pages a sequence of a paged cache holds.  Lengths come from
// device memory and may be anything: no sum here leaves 32 bits (len + page - 1
// would, for lengths within a page of 2^31).  Plain C++, so that the host tests
// compile it too.
#pragma once

#ifdef __CUDACC__
#define ATTN_PAGES_FN __host__ __device__ __forceinline__
#else
#define ATTN_PAGES_FN inline
#endif

namespace attn {

// Pages of 2^page_log2 tokens that len >= 0 tokens take.
ATTN_PAGES_FN int pages_of(int len, int page_log2) {
  return (len >> page_log2) + ((len & ((1 << page_log2) - 1)) != 0 ? 1 : 0);
}

// Entries of its table row that a sequence holds, whatever its length says.
ATTN_PAGES_FN int held_pages(int len, int page_log2, int max_pages) {
  const int n = len > 0 ? pages_of(len, page_log2) : 0;
  return n < max_pages ? n : max_pages;
}

}  // namespace attn
