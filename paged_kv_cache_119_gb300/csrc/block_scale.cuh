// block_scale.cuh -- E4M3 caches with a scale for each block and kv head (mode kBlock of the
// attention kernels): value = code * scale[block][head], one array of scales for K, one for V.
//
// With s_t, u_t the K and V scale of token t's block and x_t its score (base 2), the output is
//     sum_t p_t u_t c_t / sum_t p_t,   p_t = 2^(x_t - m),  x_t = (q . k codes) s_t.
// The V scale rides on the exponent: with w_t = 2^(x_t + log2 u_t - M), M the largest exponent,
//     O = sum w_t c_t,   l = sum w_t / u_t,   out = O / l,
// so the kernels' online softmax runs on x_t + log2 u_t (one multiply-add where there was a
// multiply), P . V takes w_t <= 1 and the codes as they are, and only the row sums meet 1 / u_t,
// once a block.  Weights that P . V rounds in 16 or 8 bits are rounded relative to the largest
// p_t u_t, that is, to what a token can add to the output.  Scales count as held within
// 2^-48 .. 2^48: then x_t + log2 u_t - M stays above -126 for every token whose p_t is within
// 2^-30 of the largest, and the sum l loses none of them.
// Cost beside one scale a head: the loads of two floats a block, and where a CTA is bound by its
// issue slots a few percent (one scale a head / block scales: 32 x 4 new tokens of 8192, 4 heads a
// kv head, blocks of 32, 104 / 106 us; 256 rows over 4096 tokens on the chunk kernel 71.7 / 74.4;
// 8 x 32768 tokens, 64/8 heads, blocks of 16, 101 / 97).
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr float kScaleLow = 0x1p-48f, kScaleHigh = 0x1p48f;

// The scales of block e (1 where e is no block of the pool) and a head as they lie in memory,
// loaded well before they are used ...
struct RawScale {
    float k, v;
};
template <typename P>
__device__ __forceinline__ RawScale load_scale(const P& p, int e, int head)
{
    if (e < 0 || (int64_t)e >= p.num_blocks)
        return RawScale{1.f, 1.f};
    const int64_t i = (int64_t)e * p.scale_stride + head;
    return RawScale{__ldg(p.k_scale + i), __ldg(p.v_scale + i)};
}

// ... and as the kernels use them: (K scale, log2 of the V scale, its reciprocal); exact for
// powers of two.  (Together in one step, every tile of the chunk kernel waited for the loads:
// 1.43 us a tile against 0.96.)
__device__ __forceinline__ float4 block_scale(const RawScale& s)
{
    const float k = fminf(fmaxf(s.k, kScaleLow), kScaleHigh);
    const float v = fminf(fmaxf(s.v, kScaleLow), kScaleHigh);
    const int bits = __float_as_int(v);
    const float frac = __int_as_float((bits & 0x7fffff) | 0x3f800000);      // [1, 2)
    const float lg = frac == 1.f ? 0.f : log2f(frac);
    return make_float4(k, (float)((bits >> 23) - 127) + lg, __frcp_rn(v), 0.f);
}

// Scales of a CTA's blocks on their way from the producer to the consumers: block i of the CTA
// at i % kScaleRing.  The producer fills 32 entries at a time, before the copies of those
// blocks; the entries that it overwrites are of blocks more than 32 back, whose tiles are
// consumed while the ring of tiles holds at most 32 blocks.
constexpr int kScaleRing = 64;
constexpr int kScaleRingBytes = kScaleRing * 16;

}  // namespace pa
