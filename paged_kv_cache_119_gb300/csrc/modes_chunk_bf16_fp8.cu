// modes_chunk_bf16_fp8.cu -- chunk_attn_kernel's other modes, bf16 queries over E4M3 caches.
#include "modes_chunk.cuh"

namespace pa {

PA_CHUNK_MODE_FNS(bf16_fp8, __nv_bfloat16, true)

}  // namespace pa
