// tree_d128.cu -- the tree kernels for head dimension 128.
#define ATTN_TREE_D 128
#include "tree_kernel.cuh"
