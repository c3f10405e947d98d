// Instantiations of the row-tiled decode-attention kernel for bf16 and head dim 64.
#include "row_attn_kernel.cuh"
#include "row_attn_launch.cuh"

PDA_ROW_ATTN(bf16, 64, false)
