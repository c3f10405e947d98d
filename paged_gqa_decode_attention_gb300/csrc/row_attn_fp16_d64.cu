// Instantiations of the row-tiled decode-attention kernel for fp16 and head dim 64.
#include "row_attn_kernel.cuh"
#include "row_attn_launch.cuh"

PDA_ROW_ATTN(fp16, 64, true)
