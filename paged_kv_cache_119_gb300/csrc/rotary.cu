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
// Bound: HBM (read q, k, v; write q, and the k and v rows), near which the work per element
// still shows: 4096 tokens of 64 + 2 x 8 heads of 128, bf16, interleaved, 168 MB, take 34.7 us
// (4.8 TB/s), 16391 tokens of 32 + 2 x 32 heads, f16 into E4M3, 671 MB, 143 us (4.7 TB/s; the
// quotients and conversions fill the issue slots).  One CTA per token, or several that share a
// token's items when the step has few tokens: a step of 4 tokens takes 6.2 us, a launch.
#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotScales = 128;     // kv heads whose scales a CTA keeps in shared memory

// VEC elements (16 bytes, or one element) as they lie in memory
template <typename T, int VEC>
struct RotRaw {
    uint4 w;
};
template <typename T>
struct RotRaw<T, 1> {
    T w;
};

template <typename T, int VEC>
__device__ __forceinline__ RotRaw<T, VEC> rot_load(const T* p)
{
    // a plain load: q may be turned in place, so this is no read-only data
    RotRaw<T, VEC> r;
    if constexpr (VEC == 1)
        r.w = *p;
    else
        r.w = *reinterpret_cast<const uint4*>(p);
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void rot_float(const RotRaw<T, VEC>& r, float (&f)[VEC])
{
    if constexpr (VEC == 1) {
        f[0] = static_cast<float>(r.w);
    } else {
        const uint32_t u[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(u[i]);
            } else if constexpr (DType<T>::id == PA_BF16) {
                f[2 * i] = bf16_lo(u[i]);
                f[2 * i + 1] = bf16_hi(u[i]);
            } else {
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                f[2 * i] = h.x;
                f[2 * i + 1] = h.y;
            }
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void rot_store(T* p, const float (&f)[VEC])
{
    if constexpr (VEC == 1) {
        store_as(p, f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DType<T>::id == PA_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// Stores the pairs of a vector of 16-bit elements from `pairs` on as they were loaded (a NaN
// would lose its payload on the way through fp32).
template <typename T, int VEC>
__device__ __forceinline__ void rot_store_passed(T* p, const RotRaw<T, VEC>& r, int pairs)
{
    if constexpr (VEC == 8) {
        const uint32_t u[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= pairs)
                reinterpret_cast<uint32_t*>(p)[i] = u[i];
    }
}

// Quantised store: e4m3(x / scale), round to nearest even, saturating at +-448 (the codes of
// reshape_and_cache_fp8).  The fp32 quotient is the one IEEE division gives, from the correctly
// rounded reciprocal y of the scale and one remainder step (P. Markstein, IBM J. Res. Dev. 34
// (1990): with y = RN(1 / s), q = RN(x y) and the exact remainder r = x - q s, RN(q + r y) =
// RN(x / s) while nothing over- or underflows); its sign is q's (the step would lose a zero's).
// A quotient beyond 1024 saturates whatever its last bit is, and an infinite q must not meet
// its remainder: such a vector keeps its large q as they are.  An underflowing remainder
// belongs to a quotient that rounds to the code 0.  A scale whose reciprocal is not a normal
// number with room takes the division itself.
__device__ __noinline__ float rot_divide(float x, float scale) { return x / scale; }

// sc: (scale, its reciprocal, or 0 for a scale that takes the division).
__device__ __forceinline__ float2 rot_scale(float scale)
{
    const float a = fabsf(scale);
    return make_float2(scale, a >= 0x1p-100f && a <= 0x1p100f ? __frcp_rn(scale) : 0.f);
}

template <int VEC>
__device__ __forceinline__ void rot_quantise(float (&f)[VEC], float2 sc, uint32_t (&w)[(VEC + 3) / 4])
{
    if (sc.y != 0.f) {
        float big = 0.f;
        if constexpr (VEC == 1) {
            const float q = f[0] * sc.y;
            f[0] = fabsf(q) <= 1024.f ? copysignf(fmaf(fmaf(-q, sc.x, f[0]), sc.y, q), q) : q;
        } else {
            float2 q[VEC / 2];
            const float2 y2 = make_float2(sc.y, sc.y), s2 = make_float2(-sc.x, -sc.x);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 x = make_float2(f[2 * i], f[2 * i + 1]);
                q[i] = fmul2(x, y2);
                const float2 c = ffma2(ffma2(q[i], s2, x), y2, q[i]);
                big = fmaxf(big, fmaxf(fabsf(q[i].x), fabsf(q[i].y)));
                f[2 * i] = copysignf(c.x, q[i].x);
                f[2 * i + 1] = copysignf(c.y, q[i].y);
            }
            if (!(big <= 1024.f)) {
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    f[2 * i] = fabsf(q[i].x) <= 1024.f ? f[2 * i] : q[i].x;
                    f[2 * i + 1] = fabsf(q[i].y) <= 1024.f ? f[2 * i + 1] : q[i].y;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            f[i] = rot_divide(f[i], sc.x);
    }
    if constexpr (VEC == 1) {
        w[0] = __nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k], f[4 * k + 1]),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k + 2], f[4 * k + 3]),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[k] = lo | (hi << 16);
        }
    }
}

template <int VEC>
__device__ __forceinline__ void rot_store_e4m3(unsigned char* p, float (&f)[VEC], float2 sc)
{
    uint32_t w[(VEC + 3) / 4];
    rot_quantise<VEC>(f, sc, w);
    if constexpr (VEC == 1)
        *p = (unsigned char)w[0];
    else if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t*>(p) = w[0];
}

// W row vectors as codes in one store (W = 2: 16 elements of a 16-bit type).
template <typename T, int VEC, int W>
__device__ __forceinline__ void rot_store_codes(unsigned char* p, const RotRaw<T, VEC>* r, float2 sc)
{
    float f[VEC];
    if constexpr (W == 2) {
        static_assert(VEC == 8, "two vectors of eight elements");
        uint32_t lo[2], hi[2];
        rot_float<T, VEC>(r[0], f);
        rot_quantise<VEC>(f, sc, lo);
        rot_float<T, VEC>(r[1], f);
        rot_quantise<VEC>(f, sc, hi);
        *reinterpret_cast<uint4*>(p) = make_uint4(lo[0], lo[1], hi[0], hi[1]);
    } else {
        rot_float<T, VEC>(r[0], f);
        rot_store_e4m3<VEC>(p, f, sc);
    }
}

// A thread's way through items numbered (row, vector): every `step`-th item from the first,
// without a division on the way.
struct RotWalk {
    int row, vec, drow, dvec, per;
    __device__ __forceinline__ static RotWalk from(int first, int step, int per)
    {
        RotWalk w;
        w.per = per;
        w.row = first / per;
        w.vec = first - w.row * per;
        w.drow = step / per;
        w.dvec = step - w.drow * per;
        return w;
    }
    __device__ __forceinline__ void next()
    {
        row += drow;
        vec += dvec;
        if (vec >= per) {
            vec -= per;
            ++row;
        }
    }
};

// grid = (tokens, slices); slice blockIdx.y takes every gridDim.y-th group of kRotThreads
// items of the token.  VEC: elements per item vector (16 bytes), or 1 when a half-layout pair
// does not line up with 16-byte vectors (R/2 not a multiple of VEC).  The items of a token are,
// in this order, the turned ones of q and k (half layout: two vectors; interleaved: one), the
// vector of each q and k row that interleaved pairs end in, if any, the vectors of q and k past
// R, and the vectors of v; a thread loads its next item before it works on the present one.
// FIX: the turned items of a head divide kRotThreads, so a thread meets the same pairs in every
// head and keeps their cosines and sines in registers.
template <typename T, bool FP8, bool INTER, int VEC, bool FIX>
__global__ void __launch_bounds__(kRotThreads, FP8 ? 5 : INTER ? 8 : 6)
    rotary_cache_kernel(const __grid_constant__ RotaryParams p)
{
    constexpr int NP = INTER ? VEC / 2 : VEC;    // pairs of a turned item
    // (m cos, m sin) of the token's pairs, and (1, 0) past the last
    __shared__ float2 cs[kRotMaxPairs + NP];
    __shared__ int64_t slot_base;                // element of head 0 of the slot, or -1
    // E4M3: (scale, reciprocal) of the K and V heads, as far as they fit
    __shared__ float2 scales[FP8 ? 2 * kRotScales : 1];
    const int half = p.half;
    const int nv = p.head_dim / VEC;
    const int nturn = INTER ? 2 * half / VEC : half / VEC;               // turned items of a head
    const int past = INTER ? (2 * half + VEC - 1) / VEC : 2 * nturn;     // first vector past R
    const int heads = p.num_q_heads + p.num_kv_heads;
    const int step = gridDim.y * kRotThreads;
    const int first = blockIdx.y * kRotThreads + threadIdx.x;
    const int64_t head_stride = (int64_t)p.block_size * p.head_dim;      // heads of a slot
    // W vectors of a row that does not turn are one item: two where 16-bit rows become codes,
    // so that an item stores 16 bytes (head_dim is then a multiple of 16)
    constexpr int W = FP8 && VEC == 8 ? 2 : 1;
    const bool pass_wide = past % W == 0;
    const int pw = pass_wide ? W : 1;
    const RotWalk turn0 = !INTER || nturn > 0 ? RotWalk::from(first, step, nturn) : RotWalk{heads, 0, 0, 0, 1};
    const RotWalk pass0 = past < nv ? RotWalk::from(first, step, (nv - past) / pw) : RotWalk{heads, 0, 0, 0, 1};
    const RotWalk v0 = RotWalk::from(first, step, nv / W);
    if constexpr (FP8) {
        for (int i = threadIdx.x; i < 2 * min(p.num_kv_heads, kRotScales); i += kRotThreads)
            scales[i] = rot_scale((i & 1) ? p.v_scale[i >> 1] : p.k_scale[i >> 1]);
    }
    auto scale_of = [&](int h, bool of_v) -> float2 {
        return h < kRotScales ? scales[2 * h + of_v] : rot_scale((of_v ? p.v_scale : p.k_scale)[h]);
    };

    const int64_t tok = blockIdx.x;
    const T* q = static_cast<const T*>(p.q) + tok * p.q_stride;
    const T* k = static_cast<const T*>(p.k) + tok * p.k_stride;
    const T* v = static_cast<const T*>(p.v) + tok * p.v_stride;
    T* qo = static_cast<T*>(p.q_out) + tok * p.q_out_stride;
    // row of the h-th head of q then k
    auto row_of = [&](int h) -> const T* {
        return h < p.num_q_heads ? q + h * p.head_dim : k + (h - p.num_q_heads) * p.head_dim;
    };

    // the first turned item is in flight while the angles are computed
    RotWalk at = turn0;
    RotRaw<T, VEC> xa, xb;
    auto load_turned = [&](const RotWalk& w, RotRaw<T, VEC>& a, RotRaw<T, VEC>& b) {
        if (w.row < heads) {
            const T* src = row_of(w.row) + w.vec * VEC;
            a = rot_load<T, VEC>(src);
            if (!INTER)
                b = rot_load<T, VEC>(src + half);
        }
    };
    load_turned(at, xa, xb);
    for (int i = threadIdx.x; i < half + NP; i += kRotThreads) {
        float s = 0.f, c = 1.f;
        if (i < half) {
            // turns as a signed 0.64 fraction in [-1/2, 1/2); half turns = that * 2
            const int64_t n = p.positions[tok];
            const long long phase = (long long)((unsigned long long)n * p.phase[i]);
            sincospif(__ll2float_rn(phase) * 0x1p-63f, &s, &c);
            c *= p.magnitude;
            s *= p.magnitude;
        }
        cs[i] = make_float2(c, s);
    }
    if (threadIdx.x == kRotThreads - 1) {
        const int64_t slot = p.slot_mapping[tok];
        const bool bad = slot >= p.num_blocks * p.block_size;
        if (bad && blockIdx.y == 0)
            atomicOr(p.err, PA_DEVERR_SLOT);
        const int64_t blk = slot / p.block_size;
        // a padding token (slot < 0) only gets its q
        slot_base =
            slot < 0 || bad
                ? -1
                : (blk * p.num_kv_heads * p.block_size + (slot - blk * p.block_size)) * p.head_dim;
    }
    __syncthreads();
    const int64_t base = slot_base;

    // (the clamps below hold nothing back: without them the half layouts spill up to 56 bytes more)
    float2 t[NP];
    if constexpr (FIX)
#pragma unroll
        for (int i = 0; i < NP; ++i)
            t[i] = cs[min(at.vec * NP + i, half)];
    while (at.row < heads) {
        RotWalk nx = at;
        nx.next();
        RotRaw<T, VEC> na, nb;
        load_turned(nx, na, nb);
        const bool is_k = at.row >= p.num_q_heads;
        const int h = is_k ? at.row - p.num_q_heads : at.row;
        const int d = at.vec * VEC;
        if (!is_k || base >= 0) {
            if constexpr (!FIX)
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    t[i] = cs[min(at.vec * NP + i, half)];
            float a[VEC], b[VEC];
            rot_float<T, VEC>(xa, a);
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const float x0 = a[2 * i], x1 = a[2 * i + 1];
                    a[2 * i] = fmaf(x0, t[i].x, -(x1 * t[i].y));
                    a[2 * i + 1] = fmaf(x1, t[i].x, x0 * t[i].y);
                }
            } else {
                rot_float<T, VEC>(xb, b);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const float x0 = a[i], x1 = b[i];
                    a[i] = fmaf(x0, t[i].x, -(x1 * t[i].y));
                    b[i] = fmaf(x1, t[i].x, x0 * t[i].y);
                }
            }
            const int64_t cell = base + h * head_stride + d;
            if (FP8 && is_k) {
                unsigned char* dc = static_cast<unsigned char*>(p.k_cache) + cell;
                const float2 sc = scale_of(h, false);
                rot_store_e4m3<VEC>(dc, a, sc);
                if constexpr (!INTER)
                    rot_store_e4m3<VEC>(dc + half, b, sc);
            } else {
                T* dst = is_k ? static_cast<T*>(p.k_cache) + cell : qo + h * p.head_dim + d;
                rot_store<T, VEC>(dst, a);
                if constexpr (!INTER)
                    rot_store<T, VEC>(dst + half, b);
            }
        }
        at = nx;
        xa = na;
        xb = nb;
    }

    if constexpr (INTER) {
        // the vector that R ends in: its first `pairs` pairs turn, the others pass as they are
        const int pairs = half - nturn * NP;
        if (pairs > 0)
            for (int row = first; row < heads; row += step) {
                const bool is_k = row >= p.num_q_heads;
                if (is_k && base < 0)
                    continue;
                const int h = is_k ? row - p.num_q_heads : row;
                const int d = nturn * VEC;
                const RotRaw<T, VEC> x = rot_load<T, VEC>(row_of(row) + d);
                float a[VEC];
                rot_float<T, VEC>(x, a);
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    if (i < pairs) {
                        const float2 r = cs[nturn * NP + i];
                        const float x0 = a[2 * i], x1 = a[2 * i + 1];
                        a[2 * i] = fmaf(x0, r.x, -(x1 * r.y));
                        a[2 * i + 1] = fmaf(x1, r.x, x0 * r.y);
                    }
                const int64_t cell = base + h * head_stride + d;
                if (FP8 && is_k) {
                    rot_store_e4m3<VEC>(static_cast<unsigned char*>(p.k_cache) + cell, a, scale_of(h, false));
                } else {
                    T* dst = is_k ? static_cast<T*>(p.k_cache) + cell : qo + h * p.head_dim + d;
                    rot_store<T, VEC>(dst, a);
                    rot_store_passed<T, VEC>(dst, x, pairs);
                }
            }
    }

    // Vectors that do not turn, bit for bit (or quantised): those of q and k past R, then
    // v's; the next item's loads are issued before the present one is worked on.
    auto keep = [&](auto w, const RotRaw<T, VEC>* r, int h, int d, bool to_q, bool of_v) {
        if (!to_q && base < 0)
            return;
        const int64_t cell = base + h * head_stride + d;
        if constexpr (FP8) {
            if (!to_q) {
                rot_store_codes<T, VEC, w.value>(
                    static_cast<unsigned char*>(of_v ? p.v_cache : p.k_cache) + cell, r, scale_of(h, of_v));
                return;
            }
        }
        T* dst = to_q ? qo + h * p.head_dim + d : static_cast<T*>(of_v ? p.v_cache : p.k_cache) + cell;
#pragma unroll
        for (int j = 0; j < w.value; ++j)
            *reinterpret_cast<std::remove_cv_t<std::remove_reference_t<decltype(r[j].w)>>*>(dst + j * VEC) =
                r[j].w;
    };
    auto keep_rows = [&](auto w, RotWalk it, int count, int from, auto row, auto put) {
        RotRaw<T, VEC> x[w.value], y[w.value];
        auto load_row = [&](const RotWalk& i, RotRaw<T, VEC>* r) {
            if (i.row < count) {
                const T* src = row(i.row) + (from + i.vec * w.value) * VEC;
#pragma unroll
                for (int j = 0; j < w.value; ++j)
                    r[j] = rot_load<T, VEC>(src + j * VEC);
            }
        };
        load_row(it, x);
        while (it.row < count) {
            RotWalk nx = it;
            nx.next();
            load_row(nx, y);
            put(w, x, it.row, (from + it.vec * w.value) * VEC);
            it = nx;
#pragma unroll
            for (int j = 0; j < w.value; ++j)
                x[j] = y[j];
        }
    };
    constexpr std::integral_constant<int, W> wide{};
    constexpr std::integral_constant<int, 1> one{};
    auto put_qk = [&](auto w, const RotRaw<T, VEC>* r, int row, int d) {
        const bool is_k = row >= p.num_q_heads;
        keep(w, r, is_k ? row - p.num_q_heads : row, d, !is_k, false);
    };
    if (pass_wide)
        keep_rows(wide, pass0, heads, past, row_of, put_qk);
    else
        keep_rows(one, pass0, heads, past, row_of, put_qk);
    if (base >= 0)
        keep_rows(wide, v0, p.num_kv_heads, 0, [&](int h) -> const T* { return v + h * p.head_dim; },
                  [&](auto w, const RotRaw<T, VEC>* r, int row, int d) { keep(w, r, row, d, false, true); });
}

template <typename T, bool FP8, bool INTER, int VEC>
cudaError_t launch_variant(const RotaryParams& p, cudaStream_t stream)
{
    const int per = INTER ? 2 * p.half / VEC : p.half / VEC;
    const int64_t turned = (int64_t)(p.num_q_heads + p.num_kv_heads) * std::max(per, 1);
    // few tokens: a token's items are shared over CTAs until the grid holds four per SM.  (A CTA
    // that took several tokens in turn, to set up its walks once, measured slower: 155 against
    // 142 us for 16391 tokens into E4M3.)
    const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
    const int64_t most = (turned + kRotThreads - 1) / kRotThreads;
    int64_t slices = (4 * (int64_t)sms + p.num_tokens - 1) / p.num_tokens;
    slices = slices < most ? slices : most;
    const dim3 grid((unsigned)p.num_tokens, (unsigned)slices);
    if (per > 0 && kRotThreads % per == 0)
        rotary_cache_kernel<T, FP8, INTER, VEC, true><<<grid, kRotThreads, 0, stream>>>(p);
    else
        rotary_cache_kernel<T, FP8, INTER, VEC, false><<<grid, kRotThreads, 0, stream>>>(p);
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
