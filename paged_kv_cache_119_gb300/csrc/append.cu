// append.cu -- appends new tokens to E4M3 caches that keep a scale for each block and kv head
// (block_scale.cuh), with the rotary positions of q and k in the same launch.
//
// What it computes.  Sequence s brings n_s new tokens, the last of its L_s; they touch its logical
// blocks (L_s - n_s) / B .. (L_s - 1) / B.  For each touched block and head, of K and of V apart:
//   a = the largest finite |x| among the new elements (K after its rotation, in fp32),
//   s = the smallest power of two with a <= 448 s, within 2^-48 .. 2^48,
//   where the block holds earlier tokens, whose scale is s_old: s = max(s, s_old), and if that
//     is above s_old their codes become e4m3(code s_old / s),
//   the new codes are e4m3(x / s).
// A power of two costs an E4M3 code nothing (its relative precision does not depend on the
// scale), makes x / s exact, and keeps the repeated restating of a growing block exact but for
// codes that fall below 2^-6, so that tokens appended one by one and all at once agree but for
// those.
//
// Organisation.  A unit is one touched block of a sequence; its CTAs take some of its K and V
// tiles or some of its rows of q each.  One warp holds the new rows of a (block, head) tile in
// registers as they were loaded (a row is D / 16 lanes x 16 elements), finds a by shuffles,
// and converts from the registers: k and v are read once, and no atomics or second pass over
// memory decide the scale.  When every sequence brings one token (a decode step) a row group of
// D / 16 lanes serves a tile of its own.  The angles (rotary.cu's arithmetic) are computed once
// per unit into shared memory and serve the rows of q and k.
// Bound: HBM (q in and out, k and v in, codes out) for prefills, near which the work per element
// still shows: 32 prompts of 440 to 543 tokens, 64 + 2 x 8 heads of 128, bf16, 64 dims in pairs, 598
// MB: 106 us (5.6 TB/s; blocks of 32 136, whole heads in halves 109 and 150, the scalar layout 717
// and 1163); 24 x 1150 to 1500 tokens of 2 x 16 heads of 64, f16, nothing turned, 195 MB: 34 us (5.7
// TB/s).  A step is three dependent loads and a launch: 4 sequences 4.3 us, 256 of 40 + 2 x 40 heads 8.7
// (nothing turned 5.8).
#include <algorithm>
#include <type_traits>

#include "block_scale.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kAppendThreads = 256;

// How pairs lie in a row: none turn; (i, i + half) with half a multiple of 8; (2i, 2i + 1);
// (i, i + half) with any half (element by element).
enum Layout : int { kStill = 0, kHalves = 1, kPairs = 2, kScalar = 3 };

// 16 elements of a row in two vectors of eight, as they lie in memory.
struct Raw16 {
    uint4 a, b;
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float* f)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DType<T>::id == PA_BF16) {
            f[2 * i] = bf16_lo(u[i]);
            f[2 * i + 1] = bf16_hi(u[i]);
        } else {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            f[2 * i] = h.x;
            f[2 * i + 1] = h.y;
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f)
{
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
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight values as E4M3 codes, rounded to nearest even, saturating; NaN stays NaN.
__device__ __forceinline__ uint2 codes8(const float* f)
{
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k], f[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k + 2], f[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
        w[k] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// The largest finite magnitude of the packed elements in m (a running maximum of magnitudes, two
// 16-bit patterns a word: they order as the magnitudes do), or infinity when one was not finite.
template <typename T>
__device__ __forceinline__ float packed_max(uint32_t m)
{
    const uint32_t top = max(m & 0xffffu, m >> 16);
    if constexpr (DType<T>::id == PA_BF16)
        return top >= 0x7f80u ? INFINITY : __uint_as_float(top << 16);
    else
        return top >= 0x7c00u ? INFINITY : __half2float(__ushort_as_half((unsigned short)top));
}

__device__ __forceinline__ uint32_t fold_max(uint32_t m, const uint4& w)
{
    m = __vmaxu2(m, w.x & 0x7fff7fffu);
    m = __vmaxu2(m, w.y & 0x7fff7fffu);
    m = __vmaxu2(m, w.z & 0x7fff7fffu);
    return __vmaxu2(m, w.w & 0x7fff7fffu);
}

// The same of finite elements alone.
template <typename T>
__device__ __forceinline__ uint32_t fold_finite(uint32_t m, const uint4& w)
{
    constexpr uint32_t kInf = DType<T>::id == PA_BF16 ? 0x7f807f80u : 0x7c007c00u;
    const uint32_t u[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __vmaxu2(m, u[i] & __vcmpltu2(u[i], kInf));
    return m;
}

// The smallest power of two s within the scales' range with a <= 448 s (a finite, >= 0).
__device__ __forceinline__ float scale_for(float a)
{
    const int bits = __float_as_int(a);
    // a = m 2^e, m in [1, 2): 448 = 1.75 2^8
    const int e = (bits >> 23) - 127 + ((bits & 0x7fffff) > 0x600000 ? -7 : -8);
    return __int_as_float((min(max(e, -48), 48) + 127) << 23);
}

// (m cos, m sin) of pair i at a position: the angle as a 0.64 fraction of a turn (rotary.cu).
__device__ __forceinline__ float2 turn(const AppendParams& p, int64_t position, int i)
{
    const long long phase = (long long)((unsigned long long)position * p.phase[i]);
    float s, c;
    sincospif(__ll2float_rn(phase) * 0x1p-63f, &s, &c);
    return make_float2(c * p.magnitude, s * p.magnitude);
}

// A thread's way through items numbered (token, head, item of the row): every `step`-th from the
// first, without a division on the way.
struct QWalk {
    int row, t, h, j;                                 // row = t heads + h
    int drow, dt, dh, dj, per, heads;
    __device__ __forceinline__ static QWalk from(int first, int step, int per, int heads)
    {
        QWalk w;
        w.per = per;
        w.heads = heads;
        w.row = first / per;
        w.j = first - w.row * per;
        w.t = w.row / heads;
        w.h = w.row - w.t * heads;
        w.drow = step / per;
        w.dj = step - w.drow * per;
        w.dt = w.drow / heads;
        w.dh = w.drow - w.dt * heads;
        return w;
    }
    __device__ __forceinline__ void advance()
    {
        row += drow;
        t += dt;
        h += dh;
        j += dj;
        if (j >= per) {
            j -= per;
            ++row;
            ++h;
        }
        if (h >= heads) {
            h -= heads;
            ++t;
        }
    }
};

// Whether the call serves a sequence with rows q0 .. q1 - 1 and L tokens.
__device__ __forceinline__ bool append_sound(const AppendParams& p, int q0, int q1, int L, int block_size)
{
    return q0 >= 0 && q1 >= q0 && (int64_t)q1 <= p.num_tokens && q1 - q0 <= L && q1 - q0 <= p.max_query_len &&
           (int64_t)L <= p.bt_stride * block_size;
}

// Whether sequence s leaves no row before it, if it is the first, and none behind it, if the last.
__device__ __forceinline__ bool append_owned(const AppendParams& p, int s, int q0, int q1)
{
    return (s > 0 || q0 == 0) && (s < p.num_seqs - 1 || (int64_t)q1 == p.num_tokens);
}

// CTAs per SM: the rows of q want loads in flight more than K and V want registers (4096 tokens and
// more of 64 + 2 x 8 heads: 121 us with four, 133 with three); a tile of 32 rows of 128 is 64
// registers a lane.
template <int D, int B, bool ONE>
constexpr int append_ctas() { return !ONE && D * B == 4096 ? 2 : 4; }

// ONE: every sequence brings at most one token.  B: block size (ONE: of any kind).
template <typename T, int D, int B, bool ONE, int LAYOUT>
__global__ void __launch_bounds__(kAppendThreads, append_ctas<D, B, ONE>()) append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int LPR = D / 16;                       // lanes of a row
    constexpr int GROUP = ONE ? LPR : 32;             // lanes of a tile
    constexpr int RPI = GROUP / LPR;                  // rows a tile's lanes hold at a time
    constexpr int IT = ONE ? 1 : B / RPI;
    constexpr int GPC = kAppendThreads / GROUP;       // tiles a CTA works on at a time
    constexpr int TOK = ONE ? 1 : B;
    constexpr bool kTurn = LAYOUT != kStill;
    // (m cos, m sin) of pair 8 j + k of token t at [t][k][j]: a row's lanes read consecutive words
    __shared__ float2 cs[kTurn ? TOK * D / 2 : 1];

    const int lane = threadIdx.x & 31;
    const int bs = ONE ? p.block_size : B;
    // ---- the unit: sequence s, its b-th touched block
    int s, b;
    if (p.per_seq > 0) {
        s = (int)blockIdx.x / p.per_seq;
        b = (int)blockIdx.x - s * p.per_seq;
    } else {
        // a malformed query_start may leave a sequence no unit that flags it: the first CTAs' threads look
        // at a sequence each (there are 2 num_seqs units and more; a loop in one CTA cost every form 2 %)
        const int look = (int)blockIdx.x * kAppendThreads + threadIdx.x;
        if (blockIdx.y == 0 && look < p.num_seqs) {
            const int q0 = p.query_start[look], q1 = p.query_start[look + 1];
            if (!append_owned(p, look, q0, q1) || !append_sound(p, q0, q1, p.context_lens[look], bs))
                atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
        }
        // sequence i's units start at query_start[i] / B + 2 i: it touches at most n / B + 2 blocks
        int lo = 0, hi = p.num_seqs;                   // 33-way search, all lanes of each warp
        while (hi - lo > 1) {
            const int span = hi - lo;
            const int at = span <= 32 ? lo + lane : lo + (int)((int64_t)span * (lane + 1) / 33);
            const bool le = at < hi && (int64_t)(p.query_start[at] / bs) + 2 * (int64_t)at <= (int64_t)blockIdx.x;
            const int c = __popc(__ballot_sync(kFullMask, le));
            if (span <= 32) {
                lo = max(lo, lo + c - 1);
                break;
            }
            const int next = c == 32 ? hi : lo + (int)((int64_t)span * (c + 1) / 33);
            if (c > 0)
                lo = lo + (int)((int64_t)span * c / 33);
            hi = next;
        }
        s = lo;
        b = (int)((int64_t)blockIdx.x - (p.query_start[s] / bs + 2 * (int64_t)s));
    }
    const int qs0 = p.query_start[s], qs1 = p.query_start[s + 1];
    const int n = qs1 - qs0;
    const int L = p.context_lens[s];
    const bool first_cta = p.per_seq > 0 && b == 0 && blockIdx.y == 0 && threadIdx.x == 0;
    if (first_cta && !append_owned(p, s, qs0, qs1))
        atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);       // rows before the first sequence or behind the last
    if (!append_sound(p, qs0, qs1, L, bs)) {
        if (first_cta)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
        return;
    }
    const int first = L - n;                          // position of the first new token
    const int lb = first / bs + b;                    // logical block
    if (b < 0 || lb >= (L + bs - 1) / bs || n == 0)
        return;
    const int p0 = max(first, lb * bs), ntok = min(L, lb * bs + bs) - p0;
    const int r0 = p0 - lb * bs;                      // earlier tokens of the block
    const int64_t row0 = qs0 + (p0 - first);          // the first new token's row
    const int pbn = p.block_tables[(int64_t)s * p.bt_stride + lb];
    const bool have = pbn >= 0 && (int64_t)pbn < p.num_blocks;
    if (!have && threadIdx.x == 0 && blockIdx.y == 0)
        atomicOr(p.err, PA_DEVERR_BLOCK_ID);

    const int half = p.half, J = (half + 7) / 8;
    if constexpr (kTurn) {
        for (int i = threadIdx.x; i < ntok * J * 8; i += kAppendThreads) {
            const int t = i / (J * 8), k = (i - t * J * 8) / J, j = i % J;
            if (8 * j + k < half) {
                const int64_t pos = p.positions ? p.positions[row0 + t] : p0 + t;
                cs[i] = turn(p, pos, 8 * j + k);
            }
        }
        __syncthreads();
    }

    // ---- 16 elements of a row: two vectors at dims (da, db)
    const int j = lane & (LPR - 1);
    auto dims = [&](int jj, bool turned, int& da, int& db) {
        if (LAYOUT == kHalves && turned && jj < J) {
            da = 8 * jj;
            db = half + 8 * jj;
        } else if (LAYOUT == kHalves && turned) {
            da = 2 * half + 16 * (jj - J);
            db = da + 8;
        } else {
            da = 16 * jj;
            db = da + 8;
        }
    };
    // their values (fp32), turned by token t's angles; whether anything turned
    auto values = [&](const Raw16& w, int jj, int t, float (&f)[16]) -> bool {
        unpack8<T>(w.a, f);
        unpack8<T>(w.b, f + 8);
        if (!kTurn || jj >= J)
            return false;
        const float2* c = cs + t * J * 8 + jj;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (LAYOUT == kPairs && 8 * jj + k >= half)
                break;
            const float2 r = c[k * J];
            const int x = LAYOUT == kPairs ? 2 * k : k, y = LAYOUT == kPairs ? 2 * k + 1 : k + 8;
            const float x0 = f[x], x1 = f[y];
            f[x] = fmaf(x0, r.x, -(x1 * r.y));
            f[y] = fmaf(x1, r.x, x0 * r.y);
        }
        return true;
    };

    // ---- K and V tiles of the block: (head, K or V) numbered head fastest, K first
    const int tiles = 2 * p.num_kv_heads;
    const int step = p.kv_slices * GPC;
    if (have && (int)blockIdx.y < p.kv_slices) {
        const int group = threadIdx.x / GROUP;
        const int sub = (threadIdx.x % GROUP) / LPR;  // the lane's row among RPI
        for (int base = (int)blockIdx.y * GPC; base < tiles; base += step) {
            const int tile = base + group;
            const bool live = tile < tiles;           // (uniform over a tile's lanes)
            const bool is_k = tile < p.num_kv_heads;
            const int h = live ? (is_k ? tile : tile - p.num_kv_heads) : 0;
            const T* src = static_cast<const T*>(is_k ? p.k : p.v);
            const int64_t stride = is_k ? p.k_stride : p.v_stride;
            const bool turned = kTurn && is_k;
            int da, db;
            dims(j, turned, da, db);
            const int64_t cell = (int64_t)pbn * p.num_kv_heads + h;
            unsigned char* dst = (is_k ? p.k_cache : p.v_cache) + cell * bs * D;
            float* scale_at = (is_k ? p.k_scales : p.v_scales) + (int64_t)pbn * p.scale_stride + h;
            float old = r0 > 0 && live ? *scale_at : 1.f;
            Raw16 w[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = i * RPI + sub;          // the new token's number
                w[i].a = w[i].b = make_uint4(0u, 0u, 0u, 0u);
                if (live && r < ntok) {
                    const T* row = src + (row0 + r) * stride + (int64_t)h * D;
                    w[i].a = *reinterpret_cast<const uint4*>(row + da);
                    w[i].b = *reinterpret_cast<const uint4*>(row + db);
                }
            }
            // element d of a row in the scalar layout
            auto turned_scalar = [&](int i, int r, float (&f)[16]) {
                unpack8<T>(w[i].a, f);
                unpack8<T>(w[i].b, f + 8);
                const T* row = src + (row0 + r) * stride + (int64_t)h * D;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int d = 16 * j + e;
                    if (d >= 2 * half)
                        break;
                    const int pair = d < half ? d : d - half;
                    const float other = static_cast<float>(row[d < half ? d + half : d - half]);
                    const float2 c = cs[r * J * 8 + (pair & 7) * J + (pair >> 3)];
                    f[e] = d < half ? fmaf(f[e], c.x, -(other * c.y)) : fmaf(f[e], c.x, other * c.y);
                }
            };
            auto load_values = [&](int i, float (&f)[16]) {
                const int r = i * RPI + sub;
                if (LAYOUT == kScalar && turned && live && r < ntok)
                    turned_scalar(i, r, f);
                else if (LAYOUT != kScalar && turned && r < ntok)
                    values(w[i], j, r, f);
                else {
                    unpack8<T>(w[i].a, f);
                    unpack8<T>(w[i].b, f + 8);
                }
            };
            // the largest finite magnitude: of turned values in fp32, of others from the bits (ONE:
            // a warp's tiles may be of both kinds, and shuffle together)
            float amax = 0.f;
            if (ONE || turned) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    float f[16];
                    load_values(i, f);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        amax = fabsf(f[e]) < INFINITY ? fmaxf(amax, fabsf(f[e])) : amax;
                }
#pragma unroll
                for (int m = GROUP / 2; m >= 1; m >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, m));
            } else {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < IT; ++i)
                    top = fold_max(fold_max(top, w[i].a), w[i].b);
#pragma unroll
                for (int m = GROUP / 2; m >= 1; m >>= 1)
                    top = __vmaxu2(top, __shfl_xor_sync(kFullMask, top, m));
                amax = packed_max<T>(top);
                if (__any_sync(kFullMask, amax == INFINITY)) {       // some element is not finite
                    top = 0;
#pragma unroll
                    for (int i = 0; i < IT; ++i)
                        top = fold_finite<T>(fold_finite<T>(top, w[i].a), w[i].b);
#pragma unroll
                    for (int m = GROUP / 2; m >= 1; m >>= 1)
                        top = __vmaxu2(top, __shfl_xor_sync(kFullMask, top, m));
                    amax = packed_max<T>(top);
                }
            }
            float scale = scale_for(amax);
            if (r0 > 0) {
                old = fminf(fmaxf(old, kScaleLow), kScaleHigh);
                scale = fmaxf(scale, old);
            }
            if (!live)
                continue;                             // (no shuffle follows)
            if (r0 > 0 && scale > old) {
                // the earlier tokens in the new scale
                const float ratio = old / scale;
#pragma unroll 4
                for (int r = sub; r < r0; r += RPI) {
                    uint4* at = reinterpret_cast<uint4*>(dst + r * D + 16 * j);
                    const uint4 c = *at;
                    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
                    uint32_t out[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 lo = e4m3x2_to_float2(in[k]), hi = e4m3x2_to_float2(in[k] >> 16);
                        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(lo.x * ratio, lo.y * ratio),
                                                                    __NV_SATFINITE, __NV_E4M3);
                        const uint32_t b2 = __nv_cvt_float2_to_fp8x2(make_float2(hi.x * ratio, hi.y * ratio),
                                                                     __NV_SATFINITE, __NV_E4M3);
                        out[k] = a | (b2 << 16);
                    }
                    *at = make_uint4(out[0], out[1], out[2], out[3]);
                }
            }
            if ((threadIdx.x % GROUP) == 0)
                *scale_at = scale;
            // a power of two divides exactly by its reciprocal; an earlier scale of another kind
            // (not this kernel's) takes the division
            const bool exact = (__float_as_int(scale) & 0x7fffff) == 0;
            const float inv = 1.f / scale;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = i * RPI + sub;
                if (r >= ntok)
                    break;
                float f[16];
                load_values(i, f);
                if (exact) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        f[e] *= inv;
                } else {
#pragma unroll 1
                    for (int e = 0; e < 16; ++e) {
                        float x = f[0];
#pragma unroll
                        for (int k = 0; k < 15; ++k)  // (rotates f: no dynamic index)
                            f[k] = f[k + 1];
                        f[15] = x / scale;
                    }
                }
                unsigned char* out = dst + (r0 + r) * D;
                const uint2 ca = codes8(f), cb = codes8(f + 8);
                if (LAYOUT == kHalves && db != da + 8) {
                    *reinterpret_cast<uint2*>(out + da) = ca;
                    *reinterpret_cast<uint2*>(out + db) = cb;
                } else {
                    *reinterpret_cast<uint4*>(out + da) = make_uint4(ca.x, ca.y, cb.x, cb.y);
                }
            }
        }
    }

    // ---- q: the turned items of the unit's rows, J of a row, then the vectors past them
    const int q_slice = (int)blockIdx.y - p.kv_slices;
    const int q_step = ((int)gridDim.y - p.kv_slices) * kAppendThreads;
    if (kTurn && LAYOUT != kScalar && q_slice >= 0) {
        const int rows = ntok * p.num_q_heads;
        const T* q = static_cast<const T*>(p.q) + row0 * p.q_stride;
        T* qo = static_cast<T*>(p.q_out) + row0 * p.q_out_stride;
        const int first_item = q_slice * kAppendThreads + threadIdx.x;
        QWalk at = QWalk::from(first_item, q_step, J, p.num_q_heads), nx;
        const int db_off = LAYOUT == kHalves ? half : 8;          // the second vector behind the first
        const int da_mul = LAYOUT == kHalves ? 8 : 16;
        auto load = [&](const QWalk& k, Raw16& w) {
            if (k.row < rows) {
                const T* row = q + k.t * p.q_stride + k.h * D + k.j * da_mul;
                w.a = *reinterpret_cast<const uint4*>(row);
                w.b = *reinterpret_cast<const uint4*>(row + db_off);
            }
        };
        Raw16 w, next;
        load(at, w);
        while (at.row < rows) {
            nx = at;
            nx.advance();
            load(nx, next);
            float f[16];
            values(w, at.j, at.t, f);
            Raw16 out;
            out.a = pack8<T>(f);
            out.b = pack8<T>(f + 8);
            if constexpr (LAYOUT == kPairs) {
                // pairs past the last that turns, bit for bit
                const int keep = half - 8 * at.j;                 // turned pairs of the item
                if (keep < 8) {
                    uint32_t* o = reinterpret_cast<uint32_t*>(&out);
                    const uint32_t* in = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[k] = k < keep ? o[k] : in[k];
                }
            }
            T* row = qo + at.t * p.q_out_stride + at.h * D + at.j * da_mul;
            *reinterpret_cast<uint4*>(row) = out.a;
            *reinterpret_cast<uint4*>(row + db_off) = out.b;
            w = next;
            at = nx;
        }
        const int still = (D - 16 * J) / 8;                       // vectors of a row that do not turn
        if (still > 0 && (p.q_out != p.q || p.q_out_stride != p.q_stride)) {
            at = QWalk::from(first_item, q_step, still, p.num_q_heads);
            while (at.row < rows) {
                // four loads in flight
                uint4 v[4];
                QWalk k = at;
#pragma unroll
                for (int i = 0; i < 4; ++i, k.advance())
                    if (k.row < rows)
                        v[i] = *reinterpret_cast<const uint4*>(q + k.t * p.q_stride + k.h * D + 16 * J + 8 * k.j);
#pragma unroll
                for (int i = 0; i < 4; ++i, at.advance())
                    if (at.row < rows)
                        *reinterpret_cast<uint4*>(qo + at.t * p.q_out_stride + at.h * D + 16 * J + 8 * at.j) = v[i];
            }
        }
    }
    if (LAYOUT == kScalar && q_slice >= 0) {
        // a pair, or an element past the pairs, at a time (a pair's elements are read and
        // written by one thread: q may be turned in place)
        const int per = D - half;
        const int64_t items = (int64_t)ntok * p.num_q_heads * per;
        const T* q = static_cast<const T*>(p.q);
        T* qo = static_cast<T*>(p.q_out);
        for (int64_t i = (int64_t)q_slice * kAppendThreads + threadIdx.x; i < items; i += q_step) {
            const int row = (int)(i / per), e = (int)(i - (int64_t)row * per);
            const int t = row / p.num_q_heads, h = row - t * p.num_q_heads;
            const T* in = q + (row0 + t) * p.q_stride + (int64_t)h * D;
            T* out = qo + (row0 + t) * p.q_out_stride + (int64_t)h * D;
            if (e < half) {
                const float2 c = cs[t * J * 8 + (e & 7) * J + (e >> 3)];
                const float x0 = static_cast<float>(in[e]), x1 = static_cast<float>(in[e + half]);
                store_as(out + e, fmaf(x0, c.x, -(x1 * c.y)));
                store_as(out + e + half, fmaf(x1, c.x, x0 * c.y));
            } else {
                out[e + half] = in[e + half];
            }
        }
    }
}

template <typename T, int D, int B, bool ONE, int LAYOUT>
cudaError_t launch_variant(AppendParams p, int64_t units, cudaStream_t stream)
{
    constexpr int LPR = D / 16;
    constexpr int GPC = kAppendThreads / (ONE ? LPR : 32);
    // A unit's CTAs: some for its K and V tiles, others for its rows of q, each with a few rounds
    // of work; fewer rounds while the grid would not hold four CTAs per SM.  (Rounds for q cost their
    // CTA one set of angles: with 8, the prompts of the head comment took 112 us, with 16 or 32 108.)
    const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
    const int64_t tiles = (2 * (int64_t)p.num_kv_heads + GPC - 1) / GPC;
    const int64_t rows = LAYOUT == kStill ? 0
                                          : ((ONE ? 1 : B) * (int64_t)p.num_q_heads + kAppendThreads / LPR - 1) /
                                                (kAppendThreads / LPR);
    auto slices = [&](int64_t work, int64_t rounds) { return (work + rounds - 1) / rounds; };
    int64_t kv_rounds = 2, q_rounds = 16;
    while (kv_rounds > 1 && units * (slices(tiles, kv_rounds) + slices(rows, q_rounds)) < 4 * (int64_t)sms)
        kv_rounds /= 2;
    while (q_rounds > 1 && units * (slices(tiles, kv_rounds) + slices(rows, q_rounds)) < 4 * (int64_t)sms)
        q_rounds /= 2;
    p.kv_slices = (int)slices(tiles, kv_rounds);
    const int64_t all = p.kv_slices + slices(rows, q_rounds);
    if (all > 65535)
        return cudaErrorInvalidValue;
    append_kernel<T, D, B, ONE, LAYOUT>
        <<<dim3((unsigned)units, (unsigned)all), kAppendThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int D, int LAYOUT>
cudaError_t launch_sized(const AppendParams& p, int64_t units, cudaStream_t stream)
{
    if (p.max_query_len == 1)
        return launch_variant<T, D, 16, true, LAYOUT>(p, units, stream);
    return p.block_size == 16 ? launch_variant<T, D, 16, false, LAYOUT>(p, units, stream)
                              : launch_variant<T, D, 32, false, LAYOUT>(p, units, stream);
}

template <typename T, int D>
cudaError_t launch_typed(const AppendParams& p, int layout, int64_t units, cudaStream_t stream)
{
    switch (layout) {
    case kHalves: return launch_sized<T, D, kHalves>(p, units, stream);
    case kPairs: return launch_sized<T, D, kPairs>(p, units, stream);
    case kScalar: return launch_sized<T, D, kScalar>(p, units, stream);
    default: return launch_sized<T, D, kStill>(p, units, stream);
    }
}

}  // namespace

cudaError_t launch_append(AppendParams p, pa_dtype dtype, int head_dim, bool interleaved, cudaStream_t stream)
{
    // Units: per_seq blocks of every sequence, as many as max_query_len tokens can touch; where
    // that is more than twice what num_tokens can (a long prompt among decode steps), each
    // sequence's own number, found by a search of query_start (8 kv heads of 128, nothing turned:
    // 4096 tokens beside 255 steps of one 8.3 us against 60.9; 256 sequences of 5 tokens 7.6 against 6.2
    // the other way).
    const int64_t B = p.block_size;
    const int64_t per = p.max_query_len == 1 ? 1 : (p.max_query_len + B - 2) / B + 1;
    const int64_t packed = p.num_tokens / B + 2 * (int64_t)p.num_seqs;
    const bool direct = per * p.num_seqs <= 2 * packed;
    p.per_seq = direct ? (int)per : 0;
    const int64_t units = direct ? per * p.num_seqs : packed;
    if (units > INT32_MAX)
        return cudaErrorInvalidValue;
    const int layout = p.half == 0 ? kStill : interleaved ? kPairs : p.half % 8 == 0 ? kHalves : kScalar;
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(p, layout, units, stream)
                               : launch_typed<__nv_bfloat16, 64>(p, layout, units, stream);
    if (dtype == PA_F16)
        return head_dim == 128 ? launch_typed<__half, 128>(p, layout, units, stream)
                               : launch_typed<__half, 64>(p, layout, units, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pa
