// attn_merge.cuh -- merges the partial rows of the modified-score and the shared-prefix
// calls.  With per-part maxima m_k (base 2), sums l_k and normalised rows o_k:
//   M = max m_k,  w_k = 2^(m_k - M) l_k,  o = sum w_k o_k / sum w_k.
// A part that saw no visible token has m = -inf, weight 0 and a row of zeros; a poisoned part's
// row is NaN and makes the sum NaN whatever its weight (it has none when the part held no valid
// block); no visible token at all gives the sum of the zeros.
//
// The merge is launched behind its pass and starts beside the pass's last CTAs: it finds out
// whose row it has from the call's inputs, and waits for the pass before it reads a part.
// Bound: reading the parts (a few MB that the passes have just left in L2), so latency.  One
// warp per (row, head): its lanes read the (m, l) of 32 parts at once and a 16-byte piece of
// the row each, four parts in flight; the sequence or group that owns the row is found by a
// 33-way search of all lanes.  Alone and from a cold start, 6144 rows of 10 parts take 11.6 us and
// 4096 rows of 2 or 3 parts 8.4 to 9.9.  (When this form was chosen, one CTA per row with a serial
// search and serial (m, l) reads took 1.6 and 1.2 times as long.)
#pragma once

#include "decode_kernel.cuh"

namespace pa {

constexpr int kMergeWarps = 8;

// The largest i in [0, n) with start[i] <= x (0 when there is none); start non-decreasing.
// All lanes of a warp call it together.
__device__ __forceinline__ int owner_of(const int32_t* start, int n, int64_t x, int lane)
{
    int lo = 0, hi = n;                            // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int span = hi - lo;
        const int at = span <= 32 ? lo + lane : lo + (int)((int64_t)span * (lane + 1) / 33);
        const bool le = at < hi && start[at] <= x;
        const int c = __popc(__ballot_sync(kFullMask, le));   // probes at or below the answer
        if (span <= 32)
            return max(lo, lo + c - 1);
        const int next = c == 32 ? hi : lo + (int)((int64_t)span * (c + 1) / 33);
        if (c > 0)
            lo = lo + (int)((int64_t)span * c / 33);
        hi = next;
    }
    return lo;
}

// x / d for 0 <= x, 0 < d; in 32 bits where they hold x.
__device__ __forceinline__ int64_t quotient(int64_t x, int d)
{
    return x >> 32 == 0 ? (int64_t)((uint32_t)x / (uint32_t)d) : x / d;
}

// Head dims of a row one lane holds.
template <int D>
struct RowPiece {
    static constexpr int E = D / 32;
    float f[E];
};

// This lane's piece of the merged row: parts 0 .. count - 1 and second .. second + count2 - 1
// of ml [part][2] and po [part][D].
template <int D>
__device__ __forceinline__ RowPiece<D> merge_parts(const float* ml, const float* po, int count,
                                                   int second, int count2, int lane)
{
    constexpr int E = RowPiece<D>::E;
    const int n = count + count2;
    auto part = [&](int k) { return k < count ? k : second + k - count; };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32)
        M = fmaxf(M, ml[2 * part(k)]);
#pragma unroll
    for (int msk = 16; msk >= 1; msk >>= 1)
        M = fmaxf(M, __shfl_xor_sync(kFullMask, M, msk));
    RowPiece<D> num;
#pragma unroll
    for (int e = 0; e < E; ++e)
        num.f[e] = 0.f;
    float den = 0.f;
    for (int base = 0; base < n; base += 32) {
        float w = 0.f;
        if (base + lane < n) {
            const float2 v = *reinterpret_cast<const float2*>(ml + 2 * part(base + lane));
            w = v.x == -INFINITY ? 0.f : exp2f(v.x - M) * v.y;
        }
        den += w;
        const int m = min(32, n - base);
#pragma unroll 4
        for (int k = 0; k < m; ++k) {
            const float wk = __shfl_sync(kFullMask, w, k);
            float o[E];
            Load<float, E>::run(po + (int64_t)part(base + k) * D + lane * E, o);
#pragma unroll
            for (int e = 0; e < E; ++e)
                num.f[e] = fmaf(wk, o[e], num.f[e]);
        }
    }
#pragma unroll
    for (int msk = 16; msk >= 1; msk >>= 1)
        den += __shfl_xor_sync(kFullMask, den, msk);
#pragma unroll
    for (int e = 0; e < E; ++e)
        num.f[e] = den > 0.f ? num.f[e] / den : (den == 0.f ? num.f[e] : __int_as_float(0x7fc00000));
    return num;
}

template <typename T, int D>
__device__ __forceinline__ void store_piece(const DecodeParams& p, int64_t out_row, const RowPiece<D>& r,
                                            bool nan_out, int lane)
{
#pragma unroll
    for (int e = 0; e < RowPiece<D>::E; ++e)
        store_out<T>(p, out_row * D + lane * RowPiece<D>::E + e,
                     nan_out ? __int_as_float(0x7fc00000) : r.f[e]);
}

// Parts of a row whose CTA served rows R0 .. of the n rows of sequence s: those rows decide
// which tiles were read.
__device__ __forceinline__ int mod_parts(const DecodeParams& p, int s, int L, int n, int R0, int tile_tokens)
{
    const int last = min(n - 1, (R0 + p.rows_per_cta - 1) / p.group);
    const TileOrder t = seen_tiles(seen_by(p.mods, s, L, L - n + R0 / p.group, L - n + last), tile_tokens);
    const int per = p.partition_tokens / tile_tokens;
    return (t.count + per - 1) / per;
}

template <int D>
__device__ __forceinline__ RowPiece<D> merge_row(const DecodeParams& p, int64_t out_row, int parts, int lane)
{
    return merge_parts<D>(p.part_ml + out_row * p.max_parts * 2, p.part_o + out_row * p.max_parts * D, parts, 0,
                          0, lane);
}

// Modified scores: one warp per (query row, query head), head fastest.  tile_tokens: the tile
// the launch cut its list of tiles in; p.rows_per_cta as launched.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) mod_reduce_kernel(const DecodeParams p, int tile_tokens)
{
    const int lane = threadIdx.x & 31;
    const int64_t out_row = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (out_row >= p.num_rows * p.num_q_heads)
        return;
    const int64_t row = quotient(out_row, p.num_q_heads);
    const int h = (int)(out_row - row * p.num_q_heads);
    int s = (int)row, qs0 = (int)row, n = 1;
    if (p.query_start) {
        s = owner_of(p.query_start, p.num_seqs, row, lane);
        qs0 = p.query_start[s];
        n = p.query_start[s + 1] - qs0;
    }
    const int L = p.context_lens[s];
    const bool owned = row >= qs0 && row < (int64_t)qs0 + n;       // else no sequence's row: left alone
    const bool bad = L < 0 || L > p.max_context_len || (p.query_start && (n > L || n > p.max_query_len));
    int parts = 0;
    if (owned && !bad) {
        const int R = (int)(row - qs0) * p.group + h % p.group;
        parts = mod_parts(p, s, L, n, R / p.rows_per_cta * p.rows_per_cta, tile_tokens);
    }
    grid_wait_prerequisites();                     // the parts are in place
    if ((bad || !owned) && lane == 0 && h == 0)
        atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
    if (owned)
        store_piece<T, D>(p, out_row, merge_row<D>(p, out_row, parts, lane), bad, lane);
}

// The same when only the units from p.whole_units on were cut (chunk_attn_kernel): one warp per
// row of those units, rows_per_cta of them each.  (Sending every row of the call through the
// kernel above, most of them to return, took 33 us of 600 on 4 x 512 tokens of 8192, 64 heads.)
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) mod_reduce_cut_kernel(const DecodeParams p, int tile_tokens)
{
    const int lane = threadIdx.x & 31;
    // (fewer units than SMs are cut, and all units are fewer than 2^31 / 64)
    const int i = (int)blockIdx.x * kMergeWarps + (int)(threadIdx.x >> 5);
    const int per_seq = p.num_kv_heads * p.chunks;
    const int nth = i / p.rows_per_cta;
    const int unit = p.whole_units + nth;
    if (unit >= p.num_seqs * per_seq)
        return;
    const int s = unit / per_seq;
    const int y = unit - s * per_seq;
    const int kvh = y / p.chunks;
    const int R0 = (y - kvh * p.chunks) * p.rows_per_cta;
    const int R = R0 + (i - nth * p.rows_per_cta);
    const int qs0 = p.query_start[s], n = p.query_start[s + 1] - qs0;
    const int L = p.context_lens[s];
    const bool sane = qs0 >= 0 && n >= 0 && (int64_t)qs0 + n <= p.num_rows;
    const bool bad = L < 0 || L > p.max_context_len || n > L || n > p.max_query_len;
    const bool here = sane && !bad && R / p.group < n;
    const int parts = here ? mod_parts(p, s, L, n, R0, tile_tokens) : 0;
    auto out_row = [&](int r) -> int64_t {
        const int tok = r / p.group;
        return (int64_t)(qs0 + tok) * p.num_q_heads + kvh * p.group + (r - tok * p.group);
    };
    grid_wait_prerequisites();                     // the parts are in place
    if (here)
        store_piece<T, D>(p, out_row(R), merge_row<D>(p, out_row(R), parts, lane), false, lane);
    if (sane && bad && R0 == 0)                    // (flagged by the pass; rows past the bound too)
        for (int64_t r = R; r < min((int64_t)n * p.group, (int64_t)INT32_MAX); r += p.rows_per_cta)
            store_piece<T, D>(p, out_row((int)r), RowPiece<D>{}, true, lane);
}

// Shared prefix: one warp per (sequence, query head), head fastest.  The prefix pass wrote
// parts 0 .. of partitions of prefix_part tokens (0: one part), the suffix pass parts
// p.part_base .. of p.partition_tokens.  Checks what the two passes could not see together:
// every sequence belongs to exactly one group, of at most max_group sequences, whose members
// agree on the length they share.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
    prefix_reduce_kernel(const DecodeParams p, const int32_t* group_start, int num_groups,
                         int max_group, int prefix_part)
{
    const int lane = threadIdx.x & 31;
    const int64_t out_row = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (out_row >= (int64_t)p.num_seqs * p.num_q_heads)
        return;
    const int s = (int)quotient(out_row, p.num_q_heads);
    const int g = owner_of(group_start, num_groups, s, lane);
    const int g0 = group_start[g], g1 = group_start[g + 1];
    const int L = p.context_lens[s];
    const int P = p.prefix_lens[s];
    const bool in_group = g0 >= 0 && g0 <= s && s < g1 && g1 <= p.num_seqs && g1 - g0 <= max_group;
    const bool bad = !in_group || P < 0 || P > p.max_prefix_len || L < P || L > p.max_context_len ||
                     L - P > p.max_suffix_len || p.prefix_lens[in_group ? g0 : s] != P ||
                     P % p.tile_align != 0;
    RowPiece<D> out{};
    grid_wait_prerequisites();                     // the parts are in place
    if (bad) {
        if (lane == 0 && out_row == (int64_t)s * p.num_q_heads)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
    } else {
        const int npre = P == 0 ? 0 : (prefix_part > 0 ? (P + prefix_part - 1) / prefix_part : 1);
        const int own = L - P;
        const int nsuf = own == 0 ? 0
                                  : (p.partition_tokens > 0
                                         ? (own + p.partition_tokens - 1) / p.partition_tokens
                                         : 1);
        out = merge_parts<D>(p.part_ml + out_row * p.max_parts * 2, p.part_o + out_row * p.max_parts * D,
                             npre, p.part_base, nsuf, lane);
    }
    store_piece<T, D>(p, out_row, out, bad, lane);
}

}  // namespace pa
