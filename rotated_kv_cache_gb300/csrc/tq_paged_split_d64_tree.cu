// tq_paged_split_d64_tree.cu -- paged launches of the specialised split kernel at head_dim 64,
// new tokens that see one another by masks.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(64, 3, d64_tree)
