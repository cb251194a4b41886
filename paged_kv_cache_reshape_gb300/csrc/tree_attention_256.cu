// The tree attention kernels of head_size 256.
#define PA_TREE_D 256
#include "tree_attention.cuh"
