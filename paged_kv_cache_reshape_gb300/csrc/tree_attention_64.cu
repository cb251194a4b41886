// The tree attention kernels of head_size 64.
#define PA_TREE_D 64
#include "tree_attention.cuh"
