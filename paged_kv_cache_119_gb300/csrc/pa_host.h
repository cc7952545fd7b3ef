// pa_host.h -- host helpers shared by the entry points: argument checks, the split
// decisions and the workspace layout.  Not part of the C ABI.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "pa.h"
#include "pa_internal.h"

namespace pa {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t elem_size(int dt) { return dt == PA_F32 ? 4 : (dt == PA_FP8_E4M3 ? 1 : 2); }

inline bool valid_dtype(int dt) { return dt == PA_F32 || dt == PA_F16 || dt == PA_BF16; }

// [a, a + na) and [b, b + nb) share a byte.
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// Whether [ws, ws + n) shares a byte with any of the buffers: a workspace the kernels
// write while they read the call's inputs must be disjoint from all of them.
struct Span {
    const void* p;
    size_t n;
};
inline bool overlaps_any(const void* ws, size_t n, std::initializer_list<Span> bufs)
{
    for (const Span& b : bufs)
        if (overlaps(ws, n, b.p, b.n))
            return true;
    return false;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Query heads served by one decode CTA: the largest of 8, 4, 2, 1 dividing the group.
inline int heads_per_cta(int group)
{
    for (int gc : {8, 4, 2, 1})
        if (group % gc == 0)
            return gc;
    return 1;
}

// Partition length in tokens, or 0 for one pass per (sequence, kv head).
// partition_size < 0: never split; > 0: that length whenever it splits anything.
// 0 (automatic): with units = sequences x kv heads x head chunks (CTAs per
// partition) and slots = SMs x resident decode CTAs per SM, keep one pass when
// units > slots / 2 (the unsplit grid already fills at least half the GPU).
// Otherwise split into parts = min(slots / units, max_context_len / 512) so that
// one wave of CTAs fills the resident slots: concurrent CTAs share the HBM
// bandwidth, so a single full wave of long partitions beats several waves of
// short ones (measured on GB300: 8 x 32768 tokens, 64 CTAs per partition,
// 166 us at 8 parts vs 171 us at 19 and 194 us at 64).
inline int choose_partition(int partition_size, int max_context_len, int64_t units, int64_t slots,
                     int block_size)
{
    if (partition_size < 0)
        return 0;
    if (partition_size > 0)
        return max_context_len > partition_size ? partition_size : 0;
    const int pmin = kAutoPartitionTokens;
    if (max_context_len <= pmin)
        return 0;
    if (slots <= 0)
        slots = 2 * 148;
    if (2 * units > slots)
        return 0;
    const int64_t max_parts = (max_context_len + pmin - 1) / pmin;
    const int64_t parts = std::min<int64_t>(slots / units, max_parts);
    if (parts <= 1)
        return 0;
    const int per = (int)((max_context_len + parts - 1) / parts);
    const int P = (per + block_size - 1) / block_size * block_size;
    return P >= max_context_len ? 0 : P;
}

// Partition length of the chunk-attention kernel (a multiple of its 64-token K/V
// tile), or 0 for one pass; the same one-wave rule as choose_partition.
inline int choose_chunk_partition(int partition_size, int max_context_len, int64_t units, int64_t slots)
{
    if (partition_size < 0)
        return 0;
    if (partition_size > 0)
        return max_context_len > partition_size ? partition_size : 0;
    const int pmin = kAutoPartitionTokens;
    if (max_context_len <= pmin)
        return 0;
    if (slots <= 0)
        slots = 148;
    if (2 * units > slots)
        return 0;
    const int64_t max_parts = (max_context_len + pmin - 1) / pmin;
    const int64_t parts = std::min<int64_t>(slots / units, max_parts);
    if (parts <= 1)
        return 0;
    const int per = (int)((max_context_len + parts - 1) / parts);
    const int P = (per + 63) / 64 * 64;
    return P >= max_context_len ? 0 : P;
}

// Partition length of the E4M3 tensor-core decode (decode_tc8.cuh), or 0 for one pass.
// A CTA of that kernel keeps about one 32 KB tile load in flight, so the grid needs many
// CTAs to cover the memory latency: with units = CTAs per partition and slots = SMs x
// resident CTAs per SM, contexts are cut until the grid holds about four CTAs per slot,
// into whole 128-token tiles of at least 512 tokens.  An explicit partition_size is
// used as in choose_partition.
inline int choose_partition_tc8(int partition_size, int max_context_len, int64_t units, int64_t slots)
{
    if (partition_size < 0)
        return 0;
    if (partition_size > 0)
        return max_context_len > partition_size ? partition_size : 0;
    if (slots <= 0)
        slots = 3 * 148;
    const int64_t want = 4 * slots;
    if (units >= want || max_context_len <= 512)
        return 0;
    const int64_t max_parts = (max_context_len + 511) / 512;
    const int64_t parts = std::min<int64_t>((want + units - 1) / units, max_parts);
    if (parts <= 1)
        return 0;
    const int per = (int)((max_context_len + parts - 1) / parts);
    const int P = (per + 127) / 128 * 128;
    return P >= max_context_len ? 0 : P;
}

inline size_t workspace_layout(int64_t rows, int max_parts, int head_dim, size_t* ml_offset)
{
    const size_t o_bytes = align_up((size_t)rows * max_parts * head_dim * sizeof(float), 256);
    if (ml_offset)
        *ml_offset = o_bytes;
    return o_bytes + (size_t)rows * max_parts * 2 * sizeof(float);
}

}  // namespace pa
