// modes_core.cu -- decode_kernel (CUDA cores) with modified scores and over the tokens after
// a shared prefix: fp32 caches (modified scores only), one or two query heads per kv head
// over 16-bit caches, and the same over E4M3 caches at head_dim 64.
#include "decode_kernel.cuh"
#include "modes.cuh"

namespace pa {

namespace {

template <typename T, typename TK, int D, int BS, int GC, int MODE>
struct CoreMode {
    using V = CoreVariant<T, TK, D, BS, GC, MODE>;
    static constexpr int kThreads = kDecodeThreads;
    static constexpr int kSmem = V::Smem::kBytes;
    static constexpr auto kernel() { return V::kernel(); }
    static cudaError_t configure() { return V::configure(); }
};

// Calls f with the variant's type; false when it is not built.
template <typename T, typename TK, int MODE, typename F>
bool core_variant(int head_dim, int block_size, int gc, F&& f)
{
#define PA_CORE_MODE(D_, BS_, GC_)                                      \
    if (head_dim == D_ && block_size == BS_ && gc == GC_) {             \
        f(CoreMode<T, TK, D_, BS_, GC_, MODE>{});                       \
        return true;                                                    \
    }
#define PA_CORE_MODE_D(D_)                                              \
    PA_CORE_MODE(D_, 16, 1) PA_CORE_MODE(D_, 16, 2) PA_CORE_MODE(D_, 32, 1) PA_CORE_MODE(D_, 32, 2)
    PA_CORE_MODE_D(64)
    if constexpr (sizeof(TK) != 1) {
        PA_CORE_MODE_D(128)
    }
    if constexpr (sizeof(TK) == 4) {
        PA_CORE_MODE(64, 16, 4) PA_CORE_MODE(64, 16, 8) PA_CORE_MODE(64, 32, 4)
        PA_CORE_MODE(64, 32, 8) PA_CORE_MODE(128, 16, 4) PA_CORE_MODE(128, 16, 8)
        PA_CORE_MODE(128, 32, 4) PA_CORE_MODE(128, 32, 8)
    }
#undef PA_CORE_MODE_D
#undef PA_CORE_MODE
    return false;
}

template <int MODE, typename F>
bool core_typed(pa_dtype q_dtype, pa_dtype kv_dtype, int head_dim, int block_size, int gc, F&& f)
{
    const bool fp8 = kv_dtype == PA_FP8_E4M3;
    if constexpr (MODE == kMod)
        if (kv_dtype == PA_F32)
            return core_variant<float, float, MODE>(head_dim, block_size, gc, f);
    if (q_dtype == PA_BF16)
        return fp8 ? core_variant<__nv_bfloat16, __nv_fp8_e4m3, MODE>(head_dim, block_size, gc, f)
                   : core_variant<__nv_bfloat16, __nv_bfloat16, MODE>(head_dim, block_size, gc, f);
    if (q_dtype == PA_F16)
        return fp8 ? core_variant<__half, __nv_fp8_e4m3, MODE>(head_dim, block_size, gc, f)
                   : core_variant<__half, __half, MODE>(head_dim, block_size, gc, f);
    return false;
}

template <typename F>
bool core_mode(AttnMode mode, pa_dtype q_dtype, pa_dtype kv_dtype, int head_dim, int block_size, int gc,
               F&& f)
{
    return mode == kMod ? core_typed<kMod>(q_dtype, kv_dtype, head_dim, block_size, gc, f)
                        : core_typed<kSuffix>(q_dtype, kv_dtype, head_dim, block_size, gc, f);
}

}  // namespace

cudaError_t launch_core_mode(const DecodeParams& p, AttnMode mode, pa_dtype q_dtype, pa_dtype kv_dtype,
                             int head_dim, int block_size, int gc, dim3 grid, cudaStream_t stream)
{
    cudaError_t err = cudaErrorInvalidValue;
    core_mode(mode, q_dtype, kv_dtype, head_dim, block_size, gc,
              [&](auto v) { err = launch_mode_variant<decltype(v)>(grid, stream, p); });
    return err;
}

int occupancy_core_mode(AttnMode mode, pa_dtype q_dtype, pa_dtype kv_dtype, int head_dim, int block_size,
                        int gc)
{
    int n = 0;
    core_mode(mode, q_dtype, kv_dtype, head_dim, block_size, gc,
              [&](auto v) { n = occupancy_mode_variant<decltype(v)>(); });
    return n;
}

}  // namespace pa
