// rotary.cu -- rotary positions fused with the cache write: one launch turns the rows of
// q and k by their positions, stores q, and writes the turned k and the v rows to the
// cache slots slot_mapping names (as reshape_and_cache does for rows that are ready).
//
// Mathematics.  Pair i < R/2 of a head row at position n turns by the angle n f_i:
//     y_a = m (x_a cos - x_b sin),   y_b = m (x_b cos + x_a sin),
// with (a, b) = (i, i + R/2), or (2i, 2i + 1) for interleaved pairs; dims >= R pass.
//   * Angles.  n f_i grows to 10^5 radians and more, where a fp32 product has lost the
//     fraction of a turn.  The host turns f_i into turns per position as a 0.64 fixed-point
//     fraction F_i = round(f_i / 2 pi * 2^64) mod 2^64, and the kernel multiplies modulo
//     2^64: the wrap drops the whole turns, so the phase is exact to |n| 2^-65 turns for
//     every int32 position, with one 64-bit integer product and no fp64.  sincospif then
//     sees half turns in [-1, 1].
//   * The R/2 (cos, sin) pairs of a token are shared by its heads: the CTA computes them
//     once into shared memory (magnitude folded in), then its threads run over the
//     (head, 16-byte vector) items.  A half-layout item is the two vectors i .. and
//     i + R/2 .., so that every element is read once; the arithmetic is fp32 and each
//     result is rounded once, to the row type or, divided by the head's scale, to E4M3.
// Bound: HBM (read q, k, v; write q, and the k and v rows); one CTA per token, or several
// that share a token's items when the step has few tokens.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRotThreads = 256;

// VEC elements (VEC * sizeof(T) = 16 bytes, or one element) as fp32
template <typename T, int VEC>
struct RotVec {
    float f[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ RotVec<T, VEC> rot_load(const T* p)
{
    RotVec<T, VEC> r;
    if constexpr (VEC == 1) {
        r.f[0] = static_cast<float>(*p);
    } else {
        // a plain load: q may be turned in place, so this is no read-only data
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.f[i] = __uint_as_float(u[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DType<T>::id == PA_BF16) {
                    r.f[2 * i] = bf16_lo(u[i]);
                    r.f[2 * i + 1] = bf16_hi(u[i]);
                } else {
                    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                    r.f[2 * i] = h.x;
                    r.f[2 * i + 1] = h.y;
                }
            }
        }
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void rot_store(T* p, const RotVec<T, VEC>& r)
{
    if constexpr (VEC == 1) {
        store_as(p, r.f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(r.f[0], r.f[1], r.f[2], r.f[3]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DType<T>::id == PA_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(r.f[2 * i], r.f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(r.f[2 * i], r.f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// Quantised store: e4m3(x / scale), IEEE division, round to nearest even, saturating at
// +-448 (the codes of reshape_and_cache_fp8).
template <typename T, int VEC>
__device__ __forceinline__ void rot_store_e4m3(unsigned char* p, const RotVec<T, VEC>& r, float scale)
{
    if constexpr (VEC == 1) {
        *p = (unsigned char)__nv_cvt_float_to_fp8(r.f[0] / scale, __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(r.f[4 * k] / scale, r.f[4 * k + 1] / scale), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(r.f[4 * k + 2] / scale, r.f[4 * k + 3] / scale), __NV_SATFINITE, __NV_E4M3);
            w[k] = lo | (hi << 16);
        }
        if constexpr (VEC == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

// grid = (tokens, slices); slice blockIdx.y takes every gridDim.y-th group of
// kRotThreads items of the token.  VEC: elements per item vector (16 bytes), or 1 when a
// half-layout pair does not line up with 16-byte vectors (R/2 not a multiple of VEC).
template <typename T, bool FP8, bool INTER, int VEC>
__global__ void __launch_bounds__(kRotThreads) rotary_cache_kernel(const __grid_constant__ RotaryParams p)
{
    __shared__ float2 cs[kRotMaxPairs];          // (m cos, m sin) of the token's pairs
    const int64_t tok = blockIdx.x;
    const int half = p.half;
    const int64_t slot = p.slot_mapping[tok];
    const int64_t n = p.positions[tok];
    for (int i = threadIdx.x; i < half; i += kRotThreads) {
        // turns as a signed 0.64 fraction in [-1/2, 1/2); half turns = that * 2
        const long long phase = (long long)((unsigned long long)n * p.phase[i]);
        float s, c;
        sincospif(__ll2float_rn(phase) * 0x1p-63f, &s, &c);
        cs[i] = make_float2(c * p.magnitude, s * p.magnitude);
    }
    const bool bad_slot = slot >= p.num_blocks * p.block_size;
    if (bad_slot && threadIdx.x == 0 && blockIdx.y == 0)
        atomicOr(p.err, PA_DEVERR_SLOT);
    const bool write = slot >= 0 && !bad_slot;   // a padding token only gets its q
    const int64_t blk = write ? slot / p.block_size : 0;
    const int64_t off = write ? slot - blk * p.block_size : 0;
    // element of head 0 of the slot; heads lie block_size * head_dim apart
    const int64_t base = (blk * p.num_kv_heads * p.block_size + off) * p.head_dim;
    const int64_t head_stride = (int64_t)p.block_size * p.head_dim;
    __syncthreads();

    // items of a turned head: half-layout pairs of vectors then the vectors past R, or,
    // interleaved, its vectors
    const int nv = p.head_dim / VEC;
    const int npair = INTER ? 0 : half / VEC;
    const int per_head = nv - npair;
    const int turned = (p.num_q_heads + p.num_kv_heads) * per_head;
    const int q_items = p.num_q_heads * per_head;
    const int total = write ? turned + p.num_kv_heads * nv : q_items;
    const T* q = static_cast<const T*>(p.q) + tok * p.q_stride;
    const T* k = static_cast<const T*>(p.k) + tok * p.k_stride;
    const T* v = static_cast<const T*>(p.v) + tok * p.v_stride;
    T* qo = static_cast<T*>(p.q_out) + tok * p.q_out_stride;

    for (int item = blockIdx.y * kRotThreads + threadIdx.x; item < total;
         item += gridDim.y * kRotThreads) {
        if (item >= turned) {                    // a vector of v
            const int j = item - turned;
            const int h = j / nv;
            const int d = (j - h * nv) * VEC;
            const int64_t dst = base + h * head_stride + d;
            if constexpr (FP8) {
                rot_store_e4m3<T, VEC>(static_cast<unsigned char*>(p.v_cache) + dst,
                                       rot_load<T, VEC>(v + h * p.head_dim + d), p.v_scale[h]);
            } else if constexpr (VEC == 1) {     // bit for bit, as reshape_and_cache
                static_cast<T*>(p.v_cache)[dst] = v[h * p.head_dim + d];
            } else {
                *reinterpret_cast<uint4*>(static_cast<T*>(p.v_cache) + dst) =
                    *reinterpret_cast<const uint4*>(v + h * p.head_dim + d);
            }
            continue;
        }
        const int hh = item / per_head;          // q heads, then k heads
        const int w = item - hh * per_head;
        const bool is_k = hh >= p.num_q_heads;
        const int h = is_k ? hh - p.num_q_heads : hh;
        const T* src = (is_k ? k : q) + h * p.head_dim;
        const int da = w < npair ? w * VEC : (w + npair) * VEC;
        RotVec<T, VEC> a = rot_load<T, VEC>(src + da), b;
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const int pr = (da + i) >> 1;
                if (pr < half) {
                    const float2 t = cs[pr];
                    const float xa = a.f[i], xb = a.f[i + 1];
                    a.f[i] = fmaf(xa, t.x, -(xb * t.y));
                    a.f[i + 1] = fmaf(xb, t.x, xa * t.y);
                }
            }
        } else if (w < npair) {
            b = rot_load<T, VEC>(src + half + da);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float2 t = cs[da + i];
                const float xa = a.f[i], xb = b.f[i];
                a.f[i] = fmaf(xa, t.x, -(xb * t.y));
                b.f[i] = fmaf(xb, t.x, xa * t.y);
            }
        }
        const bool pair = !INTER && w < npair;
        if (!is_k) {
            rot_store<T, VEC>(qo + h * p.head_dim + da, a);
            if (pair)
                rot_store<T, VEC>(qo + h * p.head_dim + half + da, b);
        } else {
            const int64_t dst = base + h * head_stride + da;
            if constexpr (FP8) {
                unsigned char* kc = static_cast<unsigned char*>(p.k_cache) + dst;
                const float scale = p.k_scale[h];
                rot_store_e4m3<T, VEC>(kc, a, scale);
                if (pair)
                    rot_store_e4m3<T, VEC>(kc + half, b, scale);
            } else {
                T* kc = static_cast<T*>(p.k_cache) + dst;
                rot_store<T, VEC>(kc, a);
                if (pair)
                    rot_store<T, VEC>(kc + half, b);
            }
        }
    }
}

template <typename T, bool FP8, bool INTER, int VEC>
cudaError_t launch_variant(const RotaryParams& p, cudaStream_t stream)
{
    const int nv = p.head_dim / VEC;
    const int per_head = nv - (INTER ? 0 : p.half / VEC);
    const int64_t items =
        (int64_t)(p.num_q_heads + p.num_kv_heads) * per_head + (int64_t)p.num_kv_heads * nv;
    // few tokens: share a token's items over CTAs until the grid holds four per SM
    const int sms = device_sm_count();
    const int64_t most = (items + kRotThreads - 1) / kRotThreads;
    int64_t slices = (4 * (int64_t)(sms > 0 ? sms : 152) + p.num_tokens - 1) / p.num_tokens;
    slices = slices < most ? slices : most;
    rotary_cache_kernel<T, FP8, INTER, VEC>
        <<<dim3((unsigned)p.num_tokens, (unsigned)slices), kRotThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, bool FP8>
cudaError_t launch_typed(const RotaryParams& p, bool interleaved, cudaStream_t stream)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    if (interleaved)
        return launch_variant<T, FP8, true, VEC>(p, stream);
    if (p.half % VEC == 0)
        return launch_variant<T, FP8, false, VEC>(p, stream);
    return launch_variant<T, FP8, false, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, pa_dtype dtype, bool fp8, bool interleaved,
                          cudaStream_t stream)
{
    switch (dtype) {
    case PA_F32:
        return fp8 ? launch_typed<float, true>(p, interleaved, stream)
                   : launch_typed<float, false>(p, interleaved, stream);
    case PA_F16:
        return fp8 ? launch_typed<__half, true>(p, interleaved, stream)
                   : launch_typed<__half, false>(p, interleaved, stream);
    case PA_BF16:
        return fp8 ? launch_typed<__nv_bfloat16, true>(p, interleaved, stream)
                   : launch_typed<__nv_bfloat16, false>(p, interleaved, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
