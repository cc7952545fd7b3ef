// modes_rows_f16_fp8.cu -- decode_mma_kernel's other modes, f16 queries over E4M3 caches.
#include "modes_rows.cuh"

namespace pa {

PA_ROWS_MODE_FNS(f16_fp8, __half, __nv_fp8_e4m3)

}  // namespace pa
