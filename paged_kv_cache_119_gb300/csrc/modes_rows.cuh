// modes_rows.cuh -- decode_mma_kernel (mma.sync; 4 or 8 rows of a kv head per CTA) and
// decode_rows_kernel (16, 32 or 64) in the other modes; instantiated per query and cache type
// by modes_rows_*.cu.
#pragma once

#include "decode_mma.cuh"
#include "decode_rows.cuh"
#include "modes.cuh"

namespace pa {

// Up to 8 rows per CTA on decode_mma_kernel, 16, 32 or 64 on decode_rows_kernel.
template <typename T, typename TK, int D, int BS, int NH, int MODE>
struct RowsMode {
    static constexpr int kBPT = mma_blocks_per_tile<TK, D, BS>();
    // a row kernel's 32-token tiles: four stages (64 KB over 16-bit caches at head_dim 128)
    static constexpr int kStages = NH <= 8 ? MmaStages<TK, D, BS * kBPT>::value : kDecodeConsumerWarps;
    static constexpr int kThreads = kDecodeThreads;
    static constexpr int smem_bytes()
    {
        if constexpr (NH <= 8)
            return MmaSmem<TK, D, BS * kBPT, kStages>::kAlloc;
        else
            return RowsSmem<TK, D, kStages, NH / kRowsGroup>::kAlloc;
    }
    static constexpr int kSmem = smem_bytes();
    static constexpr auto kernel()
    {
        if constexpr (NH <= 8)
            return decode_mma_kernel<T, TK, D, BS, NH, kStages, true, kBPT, MODE>;
        else
            return decode_rows_kernel<T, TK, D, BS, kStages, MODE, NH / kRowsGroup>;
    }
    static cudaError_t configure()
    {
        return configure_once(reinterpret_cast<const void*>(kernel()), kSmem);
    }
};

// Calls f with the variant's type; false when it is not built (E4M3 caches at head_dim 128
// take 4 rows on decode_tc8_kernel, at head_dim 64 no more than 8).
template <typename T, typename TK, int MODE, typename F>
bool rows_variant(int head_dim, int block_size, int nh, F&& f)
{
#define PA_ROWS_MODE(D_, BS_, NH_)                                      \
    if (head_dim == D_ && block_size == BS_ && nh == NH_) {             \
        f(RowsMode<T, TK, D_, BS_, NH_, MODE>{});                       \
        return true;                                                    \
    }
    PA_ROWS_MODE(128, 16, 8) PA_ROWS_MODE(128, 32, 8) PA_ROWS_MODE(64, 16, 8) PA_ROWS_MODE(64, 32, 8)
    PA_ROWS_MODE(64, 16, 4) PA_ROWS_MODE(64, 32, 4)
    PA_ROWS_MODE(128, 16, 16) PA_ROWS_MODE(128, 32, 16) PA_ROWS_MODE(128, 16, 32) PA_ROWS_MODE(128, 32, 32)
    if constexpr (sizeof(TK) != 1) {
        PA_ROWS_MODE(128, 16, 4) PA_ROWS_MODE(128, 32, 4)
        PA_ROWS_MODE(64, 16, 16) PA_ROWS_MODE(64, 32, 16) PA_ROWS_MODE(64, 16, 32) PA_ROWS_MODE(64, 32, 32)
    }
    if constexpr (MODE != kPrefix) {               // (a shared prefix takes the chunk kernel there)
        PA_ROWS_MODE(128, 16, 64) PA_ROWS_MODE(128, 32, 64)
        if constexpr (sizeof(TK) != 1) {
            PA_ROWS_MODE(64, 16, 64) PA_ROWS_MODE(64, 32, 64)
        }
    }
#undef PA_ROWS_MODE
    return false;
}

template <typename T, typename TK, typename F>
bool rows_any_mode(AttnMode mode, int head_dim, int block_size, int nh, F&& f)
{
    if (mode == kMod)
        return rows_variant<T, TK, kMod>(head_dim, block_size, nh, f);
    if (mode == kModBoth)
        return rows_variant<T, TK, kModBoth>(head_dim, block_size, nh, f);
    if (mode == kPrefix)
        return rows_variant<T, TK, kPrefix>(head_dim, block_size, nh, f);
    return mode == kSuffix && rows_variant<T, TK, kSuffix>(head_dim, block_size, nh, f);
}

template <typename T, typename TK>
cudaError_t launch_rows_typed(const DecodeParams& p, AttnMode mode, int head_dim, int block_size, int nh,
                              const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid, cudaStream_t stream)
{
    cudaError_t err = cudaErrorInvalidValue;
    rows_any_mode<T, TK>(mode, head_dim, block_size, nh, [&](auto v) {
        err = launch_mode_variant<decltype(v)>(grid, stream, p, tk, tv);
    });
    return err;
}

template <typename T, typename TK>
int occupancy_rows_typed(AttnMode mode, int head_dim, int block_size, int nh)
{
    int n = 0;
    rows_any_mode<T, TK>(mode, head_dim, block_size, nh,
                         [&](auto v) { n = occupancy_mode_variant<decltype(v)>(); });
    return n;
}

// One definition of both functions for a (query type, cache type) pair.
#define PA_ROWS_MODE_FNS(name, T, TK)                                                              \
    cudaError_t launch_rows_##name(const DecodeParams& p, AttnMode mode, int head_dim,             \
                                   int block_size, int nh, const CUtensorMap& tk,                  \
                                   const CUtensorMap& tv, dim3 grid, cudaStream_t stream)          \
    {                                                                                              \
        return launch_rows_typed<T, TK>(p, mode, head_dim, block_size, nh, tk, tv, grid, stream);  \
    }                                                                                              \
    int occupancy_rows_##name(AttnMode mode, int head_dim, int block_size, int nh)                 \
    {                                                                                              \
        return occupancy_rows_typed<T, TK>(mode, head_dim, block_size, nh);                        \
    }

}  // namespace pa
