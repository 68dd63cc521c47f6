// tq_paged_split_d128.cu -- paged launches of the specialised split kernel at head_dim 128.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(128)
