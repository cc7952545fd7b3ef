// modes_rows_f16.cu -- decode_mma_kernel's other modes, f16 queries over f16 caches.
#include "modes_rows.cuh"

namespace pa {

PA_ROWS_MODE_FNS(f16, __half, __half)

}  // namespace pa
