// The tree attention kernels of head_size 128.
#define PA_TREE_D 128
#include "tree_attention.cuh"
