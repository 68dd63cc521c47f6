// tq_attention_generic_d256_tree.cu -- generic paged attention with masks among the new tokens, head_dim 256.
#include "tq_attention_generic.cuh"

TQ_PAGED_GENERIC_ENTRIES(256, 2, d256_tree)
