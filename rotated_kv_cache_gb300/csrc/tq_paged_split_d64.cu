// tq_paged_split_d64.cu -- paged launches of the specialised split kernel at head_dim 64.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(64)
