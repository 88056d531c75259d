// prefill_keep_d64.cu -- the prefill kernel with first tokens visible left of the window,
// head dimension 64.
#define ATTN_PREFILL_D 64
#define ATTN_PREFILL_KEEP
#include "prefill_kernel.cuh"
