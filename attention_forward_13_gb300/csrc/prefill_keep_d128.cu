// prefill_keep_d128.cu -- the prefill kernel with first tokens visible left of the window,
// head dimension 128.
#define ATTN_PREFILL_D 128
#define ATTN_PREFILL_KEEP
#include "prefill_kernel.cuh"
