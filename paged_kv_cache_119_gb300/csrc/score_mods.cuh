// score_mods.cuh -- what the attention kernels share beyond the plain causal softmax:
// modified scores (tanh cap, distance bias, window, tokens every row sees) and the tile
// order they leave to read, for decode_kernel, decode_mma_kernel, decode_rows_kernel,
// decode_tc8_kernel and chunk_attn_kernel.
//
// The score of a row at position pos and token t is, with x = scale q.k,
//     cap tanh(x / cap) - slope |pos - t|,
// and t is visible when t < glob, or t <= pos and pos - t < window.  The kernels keep scores
// in base-2 units (x log2 e), so the constants below carry that factor.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Every pass in a mode lets the launch behind it start as soon as all its CTAs have.  The two
// passes of a shared-prefix decode overlap so: neither needs the other.  The suffix grid has one
// z-slice more than sequences, whose first CTA waits for the prefix pass, so that the suffix
// grid does not complete before it and the merge, which waits for the suffix grid, sees both.
// Returns true for a CTA of that slice, which has nothing else to do.
template <int MODE>
__device__ __forceinline__ bool overlap_passes(int num_seqs)
{
    if constexpr (MODE != kPlain)
        grid_launch_dependents();
    if constexpr (MODE == kSuffix) {
        if ((int)blockIdx.z >= num_seqs) {
            if (blockIdx.x == 0 && blockIdx.y == 0)
                grid_wait_prerequisites();
            return true;
        }
    }
    return false;
}

// 1 / x on the MUFU unit (relative error about 2^-23; 1 / inf = 0).
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The capped score of x (both in base-2 units): c tanh(x / c).  Below |x / c| = 1/4 the odd
// Taylor series of tanh to y^9 (the next term is below 10^-8 of the result); above it
// 1 - 2 / (e^2y + 1), whose rounding (a few units of 2^-24 absolute) is there below 2^-20
// relative.  So the result is good to about 10^-6 relative for every cap.
__device__ __forceinline__ float cap_score(float x, const ScoreMods& m)
{
    const float y = x * m.inv_cap;
    const float z = y * y;
    float s = fmaf(z, 62.f / 2835.f, -17.f / 315.f);
    s = fmaf(s, z, 2.f / 15.f);
    s = fmaf(s, z, -1.f / 3.f);
    const float near0 = fmaf(y * z, s, y);
    const float e = ex2_approx(y * 2.885390081777927f);          // e^2y
    const float far0 = fmaf(-2.f, rcp_approx(e + 1.f), 1.f);
    return m.cap * (z < 0.0625f ? near0 : far0);
}

// The same where |x / c| <= kCapNear: tanh y = y P(y^2) with the four-term P of least relative
// error on [0, kCapNear^2] (5.5e-7), fitted numerically.
constexpr float kCapNear = 0.5f;
constexpr float kCapP0 = 0.99999946f, kCapP1 = -0.33326318f, kCapP2 = 0.13190297f, kCapP3 = -0.04440223f;
__device__ __forceinline__ float cap_score_near(float x, const ScoreMods& m)
{
    const float y = x * m.inv_cap;
    const float z = y * y;
    return x * fmaf(fmaf(fmaf(kCapP3, z, kCapP2), z, kCapP1), z, kCapP0);
}

// A distance slope in base-2 units, held within +-10^28 so that slope * distance (below 2^30) stays
// finite for every finite slope: from there on one token of distance already outweighs any score.
__device__ __forceinline__ float base2_slope(float s)
{
    return fminf(fmaxf(s * 1.4426950408889634f, -1e28f), 1e28f);
}

// Tokens some row of a set sees: [0, glob) and [lo, end), 0 <= glob <= end, lo <= end.
struct Seen {
    int glob, lo, end;
};

// What rows at positions first .. last of a sequence of L tokens see together.
__device__ __forceinline__ Seen seen_by(const ScoreMods& m, int seq, int L, int first, int last)
{
    Seen s;
    s.glob = m.global_lens ? max(0, min(min(m.global_lens[seq], m.max_global), L)) : 0;
    s.lo = m.window > 0 ? max(0, first - m.window + 1) : 0;
    s.end = max(last + 1, s.glob);
    return s;
}

// The tiles of TB tokens that hold a seen token, in order: tile i of `count` is tile
// i < pre ? i : i + gap of the context.
struct TileOrder {
    int pre, gap, count;
    __device__ __forceinline__ int operator()(int i) const { return i < pre ? i : i + gap; }
};
__device__ __forceinline__ TileOrder seen_tiles(const Seen& s, int TB)
{
    TileOrder t;
    t.pre = (s.glob + TB - 1) / TB;
    t.gap = max(0, s.lo / TB - t.pre);
    t.count = (s.end + TB - 1) / TB - t.gap;
    return t;
}

// Whether any token of [a, b) is seen.
__device__ __forceinline__ bool any_seen(const Seen& s, int a, int b)
{
    return a < s.glob || (b > s.lo && a < s.end);
}

__device__ __forceinline__ bool is_seen(const Seen& s, int t)
{
    return t < s.glob || (t >= s.lo && t < s.end);
}

// Whether every token of [a, a + n) is seen.
__device__ __forceinline__ bool tile_seen(const Seen& s, int a, int n)
{
    return a + n <= s.glob || (a >= s.lo && a + n <= s.end);
}

}  // namespace pa
