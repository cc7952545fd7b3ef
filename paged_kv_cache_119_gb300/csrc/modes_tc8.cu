// modes_tc8.cu -- decode_tc8_kernel (tcgen05 over E4M3 codes, head_dim 128, 1, 2 or 4 rows
// of a kv head per CTA) in the other modes.
#include "decode_kernel.cuh"
#include "decode_tc8.cuh"
#include "modes.cuh"

namespace pa {

namespace {

template <typename T, int BS, int R, int MODE>
struct Tc8Mode {
    static constexpr int kStages = 2;            // as in decode_tc8.cu: three CTAs fit on an SM
    using Sm = Tc8Smem<R, kStages>;
    static constexpr int kThreads = kTc8Threads;
    static constexpr int kSmem = Sm::kAlloc;
    static constexpr auto kernel() { return decode_tc8_kernel<T, BS, R, kStages, true, MODE>; }
    static cudaError_t configure()
    {
        return configure_once(reinterpret_cast<const void*>(kernel()), kSmem);
    }
};

template <typename T, int MODE, typename F>
bool tc8_variant(int block_size, int rows, F&& f)
{
#define PA_TC8_MODE(BS_, R_)                         \
    if (block_size == BS_ && rows == R_) {           \
        f(Tc8Mode<T, BS_, R_, MODE>{});              \
        return true;                                 \
    }
    PA_TC8_MODE(16, 4) PA_TC8_MODE(32, 4)
    if constexpr (MODE != kPrefix) {
        PA_TC8_MODE(16, 1) PA_TC8_MODE(16, 2) PA_TC8_MODE(32, 1) PA_TC8_MODE(32, 2)
    }
#undef PA_TC8_MODE
    return false;
}

template <typename T, typename F>
bool tc8_any_mode(AttnMode mode, int block_size, int rows, F&& f)
{
    if (mode == kMod)
        return tc8_variant<T, kMod>(block_size, rows, f);
    if (mode == kBlock)
        return tc8_variant<T, kBlock>(block_size, rows, f);
    if (mode == kPrefix)
        return tc8_variant<T, kPrefix>(block_size, rows, f);
    return mode == kSuffix && tc8_variant<T, kSuffix>(block_size, rows, f);
}

template <typename F>
bool tc8_typed(AttnMode mode, pa_dtype q_dtype, int block_size, int rows, F&& f)
{
    if (q_dtype == PA_BF16)
        return tc8_any_mode<__nv_bfloat16>(mode, block_size, rows, f);
    return q_dtype == PA_F16 && tc8_any_mode<__half>(mode, block_size, rows, f);
}

}  // namespace

cudaError_t launch_tc8_mode(const DecodeParams& p, AttnMode mode, pa_dtype q_dtype, int block_size,
                            int rows, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,
                            cudaStream_t stream)
{
    cudaError_t err = cudaErrorInvalidValue;
    tc8_typed(mode, q_dtype, block_size, rows,
              [&](auto v) { err = launch_mode_variant<decltype(v)>(grid, stream, p, tk, tv); });
    return err;
}

int occupancy_tc8_mode(AttnMode mode, pa_dtype q_dtype, int block_size, int rows)
{
    int n = 0;
    tc8_typed(mode, q_dtype, block_size, rows,
              [&](auto v) { n = occupancy_mode_variant<decltype(v)>(); });
    return n;
}

}  // namespace pa
