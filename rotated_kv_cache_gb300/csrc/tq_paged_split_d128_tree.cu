// tq_paged_split_d128_tree.cu -- paged launches of the specialised split kernel at head_dim 128,
// new tokens that see one another by masks.
#include "tq_paged_split.cuh"

TQ_PAGED_SPLIT_ENTRIES(128, 3, d128_tree)
