// Attention of drafted tokens (tq_tree_attention): the kernels of rows_attn.cu with items of one
// sequence whose rows are its drafted tokens' heads, and a mask over the tiles that hold drafted
// tokens.  A translation unit of its own, so that the other operators' kernels stay as they are and
// both compile at once.
#define TQ_ROWS_TREE
#include "rows_attn.cu"
