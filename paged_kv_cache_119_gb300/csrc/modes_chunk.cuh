// modes_chunk.cuh -- chunk_attn_kernel (tcgen05) with modified scores and over a shared
// prefix; instantiated per query and cache type by modes_chunk_*.cu.
#pragma once

#include "chunk_attn.cuh"
#include "modes.cuh"

namespace pa {

template <typename T, int D, int BS, bool F8, int MODE, int QT = 2>
struct ChunkMode {
    static constexpr int kStages = F8 ? 3 : QT == 1 ? 5 : ChunkStages<D>::value;
    static constexpr int kRaw = F8 ? 4 : 0;
    using Sm = ChunkSmem<D, kStages, kRaw, QT>;
    static constexpr int kThreads = chunk_threads<T, kRaw, MODE, QT>();
    static constexpr int kSmem = is_block(MODE) ? Sm::kAllocBlock : Sm::kAlloc;
    static_assert(chunk_ctas_per_sm(QT) * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
    static constexpr auto kernel() { return chunk_attn_kernel<T, D, BS, kStages, kRaw, MODE, QT>; }
    static cudaError_t configure()
    {
        return configure_once(reinterpret_cast<const void*>(kernel()), kSmem);
    }
};

// Calls f with the variant's type; false when it is not built (E4M3 needs head_dim 128).
template <typename T, bool F8, int MODE, int QT = 2, typename F>
bool chunk_variant(int head_dim, int block_size, F&& f)
{
#define PA_CHUNK_MODE(D_, BS_)                            \
    if (head_dim == D_ && block_size == BS_) {            \
        f(ChunkMode<T, D_, BS_, F8, MODE, QT>{});         \
        return true;                                      \
    }
    if constexpr (QT == 2) {
        PA_CHUNK_MODE(128, 16) PA_CHUNK_MODE(128, 32)
    }
    if constexpr (!F8) {
        PA_CHUNK_MODE(64, 16) PA_CHUNK_MODE(64, 32)
    }
#undef PA_CHUNK_MODE
    return false;
}

template <typename T, bool F8, typename F>
bool chunk_any_mode(AttnMode mode, int query_tiles, int head_dim, int block_size, F&& f)
{
    if constexpr (chunk_one_tile(kMod, 64, F8)) {
        if (query_tiles == 1)
            return mode == kMod && chunk_variant<T, F8, kMod, 1>(head_dim, block_size, f);
    }
    switch (mode) {
    case kMod: return chunk_variant<T, F8, kMod>(head_dim, block_size, f);
    case kModCap: return chunk_variant<T, F8, kModCap>(head_dim, block_size, f);
    case kModSlope: return chunk_variant<T, F8, kModSlope>(head_dim, block_size, f);
    case kModBoth: return chunk_variant<T, F8, kModBoth>(head_dim, block_size, f);
    default: break;
    }
    return mode == kPrefix && chunk_variant<T, F8, kPrefix>(head_dim, block_size, f);
}

template <typename T, bool F8>
cudaError_t launch_chunk_typed(const ChunkParams& p, AttnMode mode, int head_dim, int block_size,
                               const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid, cudaStream_t stream)
{
    cudaError_t err = cudaErrorInvalidValue;
    chunk_any_mode<T, F8>(mode, p.query_tiles, head_dim, block_size, [&](auto v) {
        err = launch_mode_variant<decltype(v)>(grid, stream, p, tk, tv);
    });
    return err;
}

#define PA_CHUNK_MODE_FNS(name, T, F8)                                                              \
    cudaError_t launch_chunk_##name(const ChunkParams& p, AttnMode mode, int head_dim,              \
                                    int block_size, const CUtensorMap& tk, const CUtensorMap& tv,   \
                                    dim3 grid, cudaStream_t stream)                                 \
    {                                                                                               \
        return launch_chunk_typed<T, F8>(p, mode, head_dim, block_size, tk, tv, grid, stream);      \
    }

}  // namespace pa
