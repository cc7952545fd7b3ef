// modes_rows_bf16.cu -- decode_mma_kernel's other modes, bf16 queries over bf16 caches.
#include "modes_rows.cuh"

namespace pa {

PA_ROWS_MODE_FNS(bf16, __nv_bfloat16, __nv_bfloat16)

}  // namespace pa
