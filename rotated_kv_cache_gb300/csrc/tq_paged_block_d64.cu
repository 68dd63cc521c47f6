// tq_paged_block_d64.cu -- paged attention of trees of up to 128 columns on tcgen05, head_dim 64.
#include "tq_paged_block.cuh"

TQ_PAGED_BLOCK_ENTRIES(64)
