// linear_d64.cu -- the chunked linear attention kernels for head dimension 64.
#define ATTN_LINEAR_D 64
#include "linear_kernel.cuh"
