// attn_merge.cuh -- merges the partial rows of the modified-score and the shared-prefix
// calls.  With per-part maxima m_k (base 2), sums l_k and normalised rows o_k:
//   M = max m_k,  w_k = 2^(m_k - M) l_k,  o = sum w_k o_k / sum w_k.
// A part that saw no visible token has m = -inf and weighs nothing; a poisoned part is NaN
// and makes the row NaN; no visible token at all gives 0.
#pragma once

#include "decode_kernel.cuh"

namespace pa {


// Head dim d of the merged row: parts first .. first + count - 1 of ml [part][2] and
// po [part][D], then count2 parts from second on.
template <int D>
__device__ __forceinline__ float merge_parts(const float* ml, const float* po, int first, int count,
                                             int second, int count2)
{
    float M = -INFINITY;
    for (int k = 0; k < count + count2; ++k)
        M = fmaxf(M, ml[2 * (k < count ? first + k : second + k - count)]);
    float num = 0.f, den = 0.f;
    for (int k = 0; k < count + count2; ++k) {
        const int i = k < count ? first + k : second + k - count;
        const float mk = ml[2 * i];
        const float w = mk == -INFINITY ? 0.f : exp2f(mk - M) * ml[2 * i + 1];
        num = fmaf(w, po[(int64_t)i * D], num);
        den += w;
    }
    return den > 0.f ? num / den : (den == 0.f ? 0.f : __int_as_float(0x7fc00000));
}

// Modified scores: one CTA of D threads per (query row, query head); grid = (rows, Hq).
// tile_tokens: the tile the launch cut its list of tiles in; p.rows_per_cta as launched.
template <typename T, int D>
__global__ void __launch_bounds__(D) mod_reduce_kernel(const DecodeParams p, int tile_tokens)
{
    const int64_t row = blockIdx.x;
    const int h = blockIdx.y;
    const int d = threadIdx.x;
    int s = (int)row, qs0 = (int)row, n = 1;
    if (p.query_start) {
        // the sequence owning the row: query_start[s] <= row < query_start[s + 1]
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.query_start[mid] <= row)
                lo = mid;
            else
                hi = mid;
        }
        s = lo;
        qs0 = p.query_start[s];
        n = p.query_start[s + 1] - qs0;
    }
    const int L = p.context_lens[s];
    const int64_t out_row = row * p.num_q_heads + h;
    const bool bad = L < 0 || L > p.max_context_len ||
                     (p.query_start && (row < qs0 || row >= (int64_t)qs0 + n || n > L ||
                                        n > p.max_query_len));
    float out;
    if (bad) {
        out = __int_as_float(0x7fc00000);
        if (d == 0 && h == 0)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
    } else {
        // the rows of the CTA that served this one decide which tiles it read
        const int R = (int)(row - qs0) * p.group + h % p.group;
        const int R0 = R / p.rows_per_cta * p.rows_per_cta;
        const int last = min(n - 1, (R0 + p.rows_per_cta - 1) / p.group);
        const TileOrder t =
            seen_tiles(seen_by(p.mods, s, L, L - n + R0 / p.group, L - n + last), tile_tokens);
        const int per = p.partition_tokens / tile_tokens;
        out = merge_parts<D>(p.part_ml + out_row * p.max_parts * 2,
                             p.part_o + out_row * p.max_parts * D + d, 0, (t.count + per - 1) / per, 0, 0);
    }
    store_out<T>(p, out_row * D + d, out);
}

// Shared prefix: one CTA of D threads per (sequence, query head); grid = (sequences, Hq).
// The prefix pass wrote parts 0 .. of partitions of prefix_part tokens (0: one part), the
// suffix pass parts p.part_base .. of p.partition_tokens.  Checks what the two passes could
// not see together: every sequence belongs to exactly one group, of at most max_group
// sequences, whose members agree on the length they share.
template <typename T, int D>
__global__ void __launch_bounds__(D)
    prefix_reduce_kernel(const DecodeParams p, const int32_t* group_start, int num_groups,
                         int max_group, int prefix_part)
{
    const int s = blockIdx.x;
    const int h = blockIdx.y;
    const int d = threadIdx.x;
    // the group owning s: group_start[g] <= s < group_start[g + 1]
    int lo = 0, hi = num_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (group_start[mid] <= s)
            lo = mid;
        else
            hi = mid;
    }
    const int g0 = group_start[lo], g1 = group_start[lo + 1];
    const int L = p.context_lens[s];
    const int P = p.prefix_lens[s];
    const bool in_group = g0 >= 0 && g0 <= s && s < g1 && g1 <= p.num_seqs && g1 - g0 <= max_group;
    const bool bad = !in_group || P < 0 || P > p.max_prefix_len || L < P ||
                     L > p.max_context_len ||
                     L - P > p.max_suffix_len || p.prefix_lens[in_group ? g0 : s] != P ||
                     P % p.tile_align != 0;
    const int64_t out_row = (int64_t)s * p.num_q_heads + h;
    float out;
    if (bad) {
        out = __int_as_float(0x7fc00000);
        if (d == 0 && h == 0)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
    } else {
        const int npre = P == 0 ? 0 : (prefix_part > 0 ? (P + prefix_part - 1) / prefix_part : 1);
        const int own = L - P;
        const int nsuf = own == 0 ? 0
                                  : (p.partition_tokens > 0
                                         ? (own + p.partition_tokens - 1) / p.partition_tokens
                                         : 1);
        out = merge_parts<D>(p.part_ml + out_row * p.max_parts * 2,
                             p.part_o + out_row * p.max_parts * D + d, 0, npre, p.part_base, nsuf);
    }
    store_out<T>(p, out_row * D + d, out);
}

}  // namespace pa
