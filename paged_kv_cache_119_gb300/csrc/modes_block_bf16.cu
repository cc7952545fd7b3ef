// modes_block_bf16.cu -- decode_mma_kernel, decode_rows_kernel and chunk_attn_kernel over E4M3
// caches with a scale for each block and head, bf16 queries.
#include "modes_block.cuh"

namespace pa {

PA_BLOCK_MODE_FNS(bf16, __nv_bfloat16)

}  // namespace pa
