// tq_paged_split_d64_any.cu -- paged launches of the specialised split kernel at head_dim 64,
// any number of new tokens.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(64, 2, d64_any)
