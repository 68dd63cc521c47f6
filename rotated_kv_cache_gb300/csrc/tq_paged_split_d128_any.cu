// tq_paged_split_d128_any.cu -- paged launches of the specialised split kernel at head_dim 128,
// any number of new tokens.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(128, 2, d128_any)
