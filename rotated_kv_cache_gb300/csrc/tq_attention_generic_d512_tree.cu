// tq_attention_generic_d512_tree.cu -- generic paged attention with masks among the new tokens, head_dim 512.
#include "tq_attention_generic.cuh"

TQ_PAGED_GENERIC_ENTRIES(512, 2, d512_tree)
