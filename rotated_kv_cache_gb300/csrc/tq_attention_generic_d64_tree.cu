// tq_attention_generic_d64_tree.cu -- generic paged attention with masks among the new tokens, head_dim 64.
#include "tq_attention_generic.cuh"

TQ_PAGED_GENERIC_ENTRIES(64, 2, d64_tree)
