// modes_chunk_f16.cu -- chunk_attn_kernel's other modes, f16 queries over f16 caches.
#include "modes_chunk.cuh"

namespace pa {

PA_CHUNK_MODE_FNS(f16, __half, false)

}  // namespace pa
