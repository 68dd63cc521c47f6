// tq_paged_block_d256.cu -- paged attention of trees of up to 128 columns on tcgen05, head_dim 256.
#include "tq_paged_block.cuh"

TQ_PAGED_BLOCK_ENTRIES(256)
