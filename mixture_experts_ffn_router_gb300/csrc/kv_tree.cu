// kv_tree.cu — attention of trees of drafted tokens over the paged cache: the kernel for chunks of tokens with
// the nodes' masks in the place of the causal rule, compiled by itself so that the two compile side by side.
#define KV_TREE 1
#include "kv_chunk.cu"
