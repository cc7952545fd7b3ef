// modes_chunk_f16_fp8.cu -- chunk_attn_kernel's other modes, f16 queries over E4M3 caches.
#include "modes_chunk.cuh"

namespace pa {

PA_CHUNK_MODE_FNS(f16_fp8, __half, true)

}  // namespace pa
