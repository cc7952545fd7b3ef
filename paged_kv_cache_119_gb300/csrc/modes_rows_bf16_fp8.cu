// modes_rows_bf16_fp8.cu -- decode_mma_kernel's other modes, bf16 queries over E4M3 caches.
#include "modes_rows.cuh"

namespace pa {

PA_ROWS_MODE_FNS(bf16_fp8, __nv_bfloat16, __nv_fp8_e4m3)

}  // namespace pa
