// modes_merge.cu -- launches the merges of attn_merge.cuh.
#include "attn_merge.cuh"
#include "modes.cuh"

namespace pa {

namespace {

// Calls f(T{}, head_dim as a constant) for the type store_out writes when out_f32 is not set
// (F32: whether the caller serves fp32 queries).
template <bool F32, typename F>
cudaError_t by_type(pa_dtype q_dtype, int head_dim, F&& f)
{
    if (q_dtype == PA_BF16)
        return head_dim == 128 ? f(__nv_bfloat16{}, std::integral_constant<int, 128>{})
                               : f(__nv_bfloat16{}, std::integral_constant<int, 64>{});
    if (q_dtype == PA_F16)
        return head_dim == 128 ? f(__half{}, std::integral_constant<int, 128>{})
                               : f(__half{}, std::integral_constant<int, 64>{});
    if constexpr (F32)
        return head_dim == 128 ? f(0.f, std::integral_constant<int, 128>{})
                               : f(0.f, std::integral_constant<int, 64>{});
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_mod_merge(const DecodeParams& p, pa_dtype q_dtype, int head_dim, int tile_tokens,
                             cudaStream_t stream)
{
    const bool cut = p.whole_units > 0;
    const int64_t rows = cut ? ((int64_t)p.num_seqs * p.num_kv_heads * p.chunks - p.whole_units) * p.rows_per_cta
                             : p.num_rows * p.num_q_heads;
    const int64_t ctas = (rows + kMergeWarps - 1) / kMergeWarps;
    if (ctas > INT32_MAX)
        return cudaErrorInvalidValue;
    return by_type<true>(q_dtype, head_dim, [&](auto t, auto d) {
        if constexpr (!std::is_same_v<decltype(t), float>)       // (the chunk kernel's types)
            if (cut)
                return launch_behind(mod_reduce_cut_kernel<decltype(t), d.value>, dim3((unsigned)ctas),
                                     dim3(32 * kMergeWarps), 0, true, stream, p, tile_tokens);
        return launch_behind(mod_reduce_kernel<decltype(t), d.value>, dim3((unsigned)ctas),
                             dim3(32 * kMergeWarps), 0, true, stream, p, tile_tokens);
    });
}

cudaError_t launch_prefix_merge(const DecodeParams& p, pa_dtype q_dtype, int head_dim,
                                const int32_t* group_start, int num_groups, int max_group,
                                int prefix_part, bool behind, cudaStream_t stream)
{
    const int64_t ctas = ((int64_t)p.num_seqs * p.num_q_heads + kMergeWarps - 1) / kMergeWarps;
    return by_type<false>(q_dtype, head_dim, [&](auto t, auto d) {
        return launch_behind(prefix_reduce_kernel<decltype(t), d.value>, dim3((unsigned)ctas),
                             dim3(32 * kMergeWarps), 0, behind, stream, p, group_start, num_groups,
                             max_group, prefix_part);
    });
}

}  // namespace pa
