// tq_paged_split_d128_one.cu -- paged launches of the specialised split kernel at head_dim 128,
// one new token a sequence.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(128, 1, d128_one)
