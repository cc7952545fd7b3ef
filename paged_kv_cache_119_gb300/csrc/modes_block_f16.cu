// modes_block_f16.cu -- decode_mma_kernel, decode_rows_kernel and chunk_attn_kernel over E4M3
// caches with a scale for each block and head, f16 queries.
#include "modes_block.cuh"

namespace pa {

PA_BLOCK_MODE_FNS(f16, __half)

}  // namespace pa
