// tq_paged_split_d256_tree.cu -- paged launches of the specialised split kernel at head_dim 256,
// new tokens that see one another by masks.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(256, 3, d256_tree)
