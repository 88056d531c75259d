// tree_d64.cu -- the tree kernels for head dimension 64.
#define ATTN_TREE_D 64
#include "tree_kernel.cuh"
