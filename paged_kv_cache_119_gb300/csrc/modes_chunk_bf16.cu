// modes_chunk_bf16.cu -- chunk_attn_kernel's other modes, bf16 queries over bf16 caches.
#include "modes_chunk.cuh"

namespace pa {

PA_CHUNK_MODE_FNS(bf16, __nv_bfloat16, false)

}  // namespace pa
