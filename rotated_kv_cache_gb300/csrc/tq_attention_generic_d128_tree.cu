// tq_attention_generic_d128_tree.cu -- generic paged attention with masks among the new tokens, head_dim 128.
#include "tq_attention_generic.cuh"

TQ_PAGED_GENERIC_ENTRIES(128, 2, d128_tree)
