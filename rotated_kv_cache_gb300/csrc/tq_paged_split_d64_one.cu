// tq_paged_split_d64_one.cu -- paged launches of the specialised split kernel at head_dim 64,
// one new token a sequence.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(64, 1, d64_one)
