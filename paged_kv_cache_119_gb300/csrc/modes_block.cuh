// modes_block.cuh -- the attention kernels in mode kBlock (E4M3 caches with a scale for each block
// and head); instantiated per query type by modes_block_*.cu, decode_tc8_kernel by modes_tc8.cu.
#pragma once

#include "modes_chunk.cuh"
#include "modes_rows.cuh"

namespace pa {

#define PA_BLOCK_MODE_FNS(name, T)                                                                   \
    cudaError_t launch_rows_block_##name(const DecodeParams& p, int head_dim, int block_size,        \
                                         int nh, const CUtensorMap& tk, const CUtensorMap& tv,       \
                                         dim3 grid, cudaStream_t stream)                             \
    {                                                                                                \
        cudaError_t err = cudaErrorInvalidValue;                                                     \
        rows_variant<T, __nv_fp8_e4m3, kBlock>(head_dim, block_size, nh, [&](auto v) {               \
            err = launch_mode_variant<decltype(v)>(grid, stream, p, tk, tv);                         \
        });                                                                                          \
        return err;                                                                                  \
    }                                                                                                \
    int occupancy_rows_block_##name(int head_dim, int block_size, int nh)                            \
    {                                                                                                \
        int n = 0;                                                                                   \
        rows_variant<T, __nv_fp8_e4m3, kBlock>(                                                      \
            head_dim, block_size, nh, [&](auto v) { n = occupancy_mode_variant<decltype(v)>(); });   \
        return n;                                                                                    \
    }                                                                                                \
    cudaError_t launch_chunk_block_##name(const ChunkParams& p, int head_dim, int block_size,        \
                                          const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,   \
                                          cudaStream_t stream)                                       \
    {                                                                                                \
        cudaError_t err = cudaErrorInvalidValue;                                                     \
        chunk_variant<T, true, kBlock>(head_dim, block_size, [&](auto v) {                           \
            err = launch_mode_variant<decltype(v)>(grid, stream, p, tk, tv);                         \
        });                                                                                          \
        return err;                                                                                  \
    }

}  // namespace pa
