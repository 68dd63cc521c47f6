// tq_paged_split_d256_any.cu -- paged launches of the specialised split kernel at head_dim 256,
// any number of new tokens.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(256, 2, d256_any)
