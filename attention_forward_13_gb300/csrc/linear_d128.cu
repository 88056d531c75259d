// linear_d128.cu -- the chunked linear attention kernels for head dimension 128.
#define ATTN_LINEAR_D 128
#include "linear_kernel.cuh"
