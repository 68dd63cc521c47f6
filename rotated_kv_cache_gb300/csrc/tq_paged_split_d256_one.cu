// tq_paged_split_d256_one.cu -- paged launches of the specialised split kernel at head_dim 256,
// one new token a sequence.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(256, 1, d256_one)
