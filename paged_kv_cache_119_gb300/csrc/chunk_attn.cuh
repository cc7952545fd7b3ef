// chunk_attn.cuh -- causal attention of a chunk of new query tokens per sequence
// over the paged KV cache, on the 5th-generation tensor cores (tcgen05, sm_103a).
//
// What it computes (the chunked-prefill / speculative-verification use of the
// paged cache: "PagedAttention 完全拆解", section "局限与未解决的问题" item 6;
// "PagedAttention 与 vLLM 推理加速", section "一图总结"): sequence s owns query rows
// query_start[s] .. query_start[s+1]-1; with n of them and context L, chunk token
// j sits at position L - n + j and attends to cached tokens 0 .. L - n + j, i.e.
// the softmax attention of section "背景" over that prefix, read through the
// block table.
//
// Organisation.  A CTA owns 256 (query token, query head) rows (128 with one query tile: see
// chunk_threads) that share a kv head -- TT = 256 / G consecutive chunk tokens x the G heads of the group, row
// r = token * G + head -- as two 128-row query tiles.  K and V stream through the
// block table in tiles of 64 tokens, each tile serving both query tiles:
//   S_q[128 x 64]  = Q_q[128 x D] . K^T      (tcgen05.mma kind::f16, fp32 in TMEM)
//   O_q[128 x D]  += P_q[128 x 64] . V        (P in f16, A operand read from tensor
//                                              memory; V in f16)
//   * warp 0 (producer): block-table entries and tensor-map TMA of the tile's K
//     and V boxes (64 dims x B tokens, 128-byte swizzle) into an mbarrier ring;
//   * warps 1 and 10: one thread each issues the MMAs of one query tile (warp 1 also
//     allocates all 512 tensor-memory columns): the scores of the next tile go out
//     before P.V of the current one, into a second S buffer.  Each issuer waits only
//     on its own query tile's completions, so the tensor core takes work from the
//     other while one waits;
//   * warps 2-5 (query tile 0) and 6-9 (query tile 1), one thread per row = TMEM
//     lane: read S, mask (causal within the chunk, end of context), online softmax
//     in base 2, write P back over the S buffer it came from (packed f16 pairs),
//     keep O up to date;
//   * over bf16 caches, warps 11-14 rewrite each V tile in place as f16 (below).
// The S/P buffers alternate between tiles, so the softmax of tile i+1 never waits
// for P.V of tile i; the scores of tile i+2 reuse a buffer only once P.V of tile i
// has read it.
// Two softmax warps per SM sub-partition hide each other's latency; the MUFU work
// (one exp2 per score) stays below the tensor-core time of a tile.
// Rescaling O is lazy: a row's reference maximum moves only when a tile's maximum
// exceeds it by more than 2^8 in probability, so p = 2^(x - m_ref) <= 256 and most
// tiles need no tensor-memory round trip.  O / l is exact for any reference, as O
// and l share it.
// P enters P.V as one f16 term, 2^7 p (at most 2^15, and normal down to p = 2^-21),
// rounded to nearest: up to 2^-11 relative per weight, so the output is off by at
// most 2^-11 of the largest |v| the row weighs (fp32 accumulation), a quarter of the
// bf16 output's own rounding step; one bf16 rounding of p would cost 2^-9, and a
// second (lo) term would cost as much tensor and softmax work again.  The 2^7 is
// carried by the exponent (p = 2^(x - m_ref + 7)) and cancels against the row sum.
// So V must be f16 too: f16 caches are, E4M3 caches convert to f16 anyway, and over
// bf16 caches four converter warps rewrite each V tile in place (same swizzled
// layout, bf16 -> f16 is exact for 2^-14 <= |v| <= 65280) and zero its rows past the
// range.  A value without an f16 value (|v| >= 65536, infinite or NaN) becomes
// infinite or NaN; the epilogue sets PA_DEVERR_RANGE for a row whose probabilities are
// finite but whose O is not.  K stays bf16 (the score product is bf16 x bf16).
// Over a shared prefix (kPrefix), whose result has to be the plain decode's, P enters as hi + lo
// terms of V's own type instead (2^-16 relative in bf16, 2^-22 in f16), which fill the 64 columns
// of the S buffer, and V is not converted: two products where there was one, and no converter
// warps over bf16 caches.  (1.0 -> 1.2 us a tile of 256 rows.  Modified scores keep the one term
// of the plain chunk call that they extend: with two, 4 x 512 tokens of 8192, 64/8 heads, capped,
// took 701 against 588 us.)
// Long contexts with few CTAs are split into partitions merged by
// chunk_reduce_kernel, as in the decode path.
// The epilogue reads O once its issuer's one-phase completion barrier has fired (P.V of
// the last two tiles may be pending or done in any combination when a warp gets there,
// which a wait on the per-tile parity barrier cannot tell apart).
//
// E4M3 caches (NRAW > 0, head_dim 128): the producer's TMA fills a ring of raw one-byte
// K + V tiles, and four converter warps (11-14) turn each into the f16 swizzled tiles of
// the ring above (E4M3 -> f16 is exact), then hand it to the issuers and release the raw
// slot.  The operands are f16: a bf16 query row is scaled into f16 range by a power of
// two (exact) that joins the row's score scale together with the kv head's K scale, and
// the V scale multiplies the output.  With block scales (kBlock, block_scale.cuh) a tile's scales
// follow it from the producer through the converters to the softmax warps.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "block_scale.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "score_mods.cuh"
#include "tc_device.cuh"

namespace pa {

constexpr int kChunkRows = 128;      // M of the tensor-core tile
constexpr int kChunkTileTok = 64;    // tokens per K/V tile (N of the score product)
// A CTA of QT (1 or 2) 128-row query tiles.  Warps: 0 producer, 1 tensor-memory allocator + MMA
// issuer of query tile 0, then 4 QT softmax warps, the issuer of query tile 1 if there is one,
// and over E4M3 and bf16 caches (or to zero V rows) the warps that convert tiles to f16.
template <int QT>
struct ChunkWarps {
    static_assert(QT == 1 || QT == 2, "one or two query tiles");
    static constexpr int kSoftmax = 4 * QT;
    static constexpr int kIssuer1 = 2 + kSoftmax;
    static constexpr int kConv0 = 1 + QT + kSoftmax;           // the first converter
    static constexpr int kConv = 2 * QT;
};
// Least factor of the scores over E4M3 caches.  Hidden columns are -infinity before the factor
// meets them, so it is never 0, which the product of a tiny bf16 row's power of two (2^-100 at
// least) and a tiny K scale can be.  Scores are below 2^33 before it: from here down they change
// no weight.
__device__ __forceinline__ float score_factor(float f) { return f < 0x1p-126f ? 0x1p-126f : f; }
// P.V takes P as 2^kChunkPExp p: p <= 2^8 (the lazy rescale), so 2^15 at most in f16
constexpr float kChunkPExp = 7.f;
static_assert(kChunkPExp == 7.f, "the partial rows of a shared prefix take 2^-7 off again");

// NRAW > 0 (E4M3 caches): a ring of NRAW raw one-byte K + V tiles that the converter
// warps turn into the 16-bit tiles of the NST-stage ring.
template <int D, int NST, int NRAW = 0, int QT = 2>
struct ChunkSmem {
    static constexpr int kHalves = D / 64;                       // 128-byte column groups
    static constexpr int kQHalf = kChunkRows * 128;              // 16 KB
    static constexpr int kQTile = kHalves * kQHalf;              // one 128-row query tile
    static constexpr int kKVHalf = kChunkTileTok * 128;          // 8 KB
    static constexpr int kKBytes = kHalves * kKVHalf;
    static constexpr int kStageBytes = 2 * kKBytes;              // K then V
    static constexpr int kQOff = 0;
    static constexpr int kStageOff = kQOff + QT * kQTile;
    static constexpr int kRawTile = kChunkTileTok * D;           // one E4M3 K (or V) tile
    static constexpr int kRawStage = 2 * kRawTile;
    static constexpr int kRawOff = kStageOff + NST * kStageBytes;
    static constexpr int kBarOff = kRawOff + NRAW * kRawStage;
    // full[NST], empty[NST], s_full[2][2], p_full[2][2], pv_done[2], q_full, mma_done[2],
    // v_zero, raw_full[NRAW], raw_empty[NRAW], vconv[NST]
    static constexpr int kNumBars = 3 * NST + 14 + 2 * NRAW;
    static constexpr int kOkOff = kBarOff + 8 * kNumBars;        // stage_ok[NST], raw_ok[NRAW]
    static constexpr int kSlotOff = kOkOff + 4 * (NST + NRAW);   // TMEM address
    static constexpr int kBytes = kSlotOff + 16;
    static constexpr int kAlloc = kBytes + 1024;                 // 1 KB alignment slack
    // kBlock: the scales of a tile's blocks (up to 4), of the stages, then of the raw slots
    static constexpr int kScaleOff = (kBytes + 15) / 16 * 16;
    static constexpr int kAllocBlock = kScaleOff + (NST + NRAW) * 64 + 1024;
    // tensor memory: O of query tile q at column 128 q, its two S/P buffers at
    // 128 (QT + q) and 64 on (P: f16 pairs in the first 32 columns)
    static constexpr int kTmemCols = 256 * QT;
    static constexpr int kSCol = 128 * QT;
    static_assert(D <= 128, "O must fit in 128 columns");
    static_assert(NRAW == 0 || D == 128, "E4M3 tiles need 128-byte rows");
    static_assert(kRawTile % 1024 == 0, "swizzle atoms need 1 KB alignment");
    static_assert(kAllocBlock <= 227 * 1024, "shared memory");
};

// Stages of the K/V ring: as many as fit next to the query tiles.
template <int D>
struct ChunkStages {
    static constexpr int value = D == 128 ? 5 : 8;
};

// Packs 8 outputs v[i] * mul (NaN when nan_out) as f16 (which = 1) or bf16 (2).
__device__ __forceinline__ uint4 pack_out8(const float* v, float mul, bool nan_out, int which)
{
    const float qnan = __int_as_float(0x7fc00000);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = nan_out ? qnan : v[2 * i] * mul;
        const float b = nan_out ? qnan : v[2 * i + 1] * mul;
        if (which == 1) {
            const __half2 h = __floats2half2_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Stores 32 consecutive outputs v[i] * mul (NaN when nan_out) at base + idx as
// fp32 (which = 0), f16 (1) or bf16 (2); idx is a multiple of 32.
__device__ __forceinline__ void store_row32(void* base, int64_t idx, const float (&v)[32], float mul,
                                            bool nan_out, int which)
{
    const float qnan = __int_as_float(0x7fc00000);
    if (which == 0) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(base) + idx);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dst[i] = nan_out ? make_float4(qnan, qnan, qnan, qnan)
                             : make_float4(v[4 * i] * mul, v[4 * i + 1] * mul, v[4 * i + 2] * mul,
                                           v[4 * i + 3] * mul);
        return;
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + idx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        dst[i] = pack_out8(v + 8 * i, mul, nan_out, which);
}

// max(a, b, c) in one instruction (NaN operands are ignored, as by fmaxf).
__device__ __forceinline__ float max3f(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Largest of a row's 64 scores.
__device__ __forceinline__ float row_max(const float (&s)[kChunkTileTok])
{
    float mx[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        mx[i] = s[i];
#pragma unroll
    for (int c = 8; c + 16 <= kChunkTileTok; c += 16)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mx[i] = max3f(mx[i], s[c + i], s[c + 8 + i]);
#pragma unroll
    for (int c = 8 + (kChunkTileTok - 8) / 16 * 16; c < kChunkTileTok; ++c)
        mx[c & 7] = fmaxf(mx[c & 7], s[c]);
    return max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

__device__ __forceinline__ float min3f(float a, float b, float c)
{
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two values as one word of two 16-bit ones (a in the low half), rounded to nearest, and back.
template <typename TM>
__device__ __forceinline__ uint32_t pack_pair(float a, float b)
{
    if constexpr (DType<TM>::id == PA_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <typename TM>
__device__ __forceinline__ float2 unpack_pair(uint32_t w)
{
    if constexpr (DType<TM>::id == PA_BF16)
        return make_float2(bf16_lo(w), bf16_hi(w));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Smallest (x) and largest (y) of a row's 64 scores.
__device__ __forceinline__ float2 row_range(const float (&s)[kChunkTileTok])
{
    float lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        lo[i] = hi[i] = s[i];
#pragma unroll
    for (int c = 4; c + 8 <= kChunkTileTok; c += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = max3f(hi[i], s[c + i], s[c + 4 + i]);
            lo[i] = min3f(lo[i], s[c + i], s[c + 4 + i]);
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = fmaxf(hi[i], s[kChunkTileTok - 4 + i]);
        lo[i] = fminf(lo[i], s[kChunkTileTok - 4 + i]);
    }
    return make_float2(min3f(fminf(lo[0], lo[1]), lo[2], lo[3]), max3f(fmaxf(hi[0], hi[1]), hi[2], hi[3]));
}

// Caps a row's 64 scores (s * mul in base-2 units, in place).  Rows of a warp that see the whole
// tile and stay within the cap itself (|y| <= 1, y = x / cap) take the six-term odd polynomial of
// tanh (least relative error there, 5.9e-7, fitted numerically); others cap_score (where a score
// is of a hidden token, what its slot holds chooses nothing).
__device__ __forceinline__ void cap_row(float (&s)[kChunkTileTok], float mul, const ScoreMods& m, bool whole)
{
    const float k = mul * m.inv_cap;
    bool within = whole;
    if (within) {
        const float2 mm = row_range(s);
        within = __all_sync(kFullMask, fmaxf(fabsf(mm.x), fabsf(mm.y)) * fabsf(k) <= 1.f);
    }
    if (within) {
        constexpr float q[6] = {0.99999941f, -0.33329042f, 0.13281434f, -0.05160568f, 0.01674312f, -0.00306706f};
#pragma unroll
        for (int c = 0; c < kChunkTileTok; c += 2) {
            const float2 y = fmul2(make_float2(s[c], s[c + 1]), make_float2(k, k));
            const float2 z = fmul2(y, y);
            float2 f = ffma2(z, make_float2(q[5], q[5]), make_float2(q[4], q[4]));
#pragma unroll
            for (int i = 3; i >= 0; --i)
                f = ffma2(z, f, make_float2(q[i], q[i]));
            const float2 x = fmul2(fmul2(y, make_float2(m.cap, m.cap)), f);
            s[c] = x.x;
            s[c + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int c = 0; c < kChunkTileTok; ++c)
            s[c] = cap_score(s[c] * mul, m);
    }
}

// grid = (partitions, num_kv_heads * m_tiles, num_seqs); chunk_threads() threads.  T: query /
// native output type.  Over E4M3 caches (value = code * per-kv-head scale) the
// tensor-core operands are f16: the codes convert exactly, a bf16 query row is scaled
// into f16 range by a power of two (exact), and the scales fold into the scores and
// the output.
// MODE: kPlain; kMod, modified scores: only the tiles that hold a token some row of the CTA
// sees are read, and the converter warps (over every cache type) zero the V rows of tokens no
// row sees; kPrefix, the rows of a group of sequences (query_start = the group's first one)
// over the tokens they share, partial rows only; kBlock, kMod over an E4M3 cache with a scale for
// each block (four or two in a tile).
// QT: query tiles of a CTA.  Two; for kMod over 16-bit caches at head_dim 64 also one, where two such
// CTAs fit on an SM: what a CTA does once (set-up, reading q, the first tile's latency, writing
// out: 5 us beside 0.8 a tile) then goes on under the other's tiles, and a unit is 128 rows.
// (choose_query_tiles in modes_api.cu has the rule; one tile was not tried for the other modes.)
template <typename T, int NRAW, int MODE, int QT = 2>
constexpr int chunk_threads()
{
    const bool conv =
        NRAW > 0 || (std::is_same_v<T, __nv_bfloat16> && MODE != kPrefix) || is_mod(MODE);
    return 32 * (ChunkWarps<QT>::kConv0 + (conv ? ChunkWarps<QT>::kConv : 0));
}

// kWideIO: live rows of a CTA up to which its warps write them out a row a lane.  The code that stores
// whole rows is longer and, run once a CTA, gains nothing for few rows.  A row a lane / whole rows, us,
// 152 CTAs over 256 tokens, head_dim 128, modified scores: f16, 40 rows 9.6 / 10.3 (fp32 out 10.0 /
// 11.7), 64 rows 9.9 / 10.5, 128 rows 11.0 / 10.7, 256 rows 15.6 / 12.0; E4M3 caches, 40 rows 11.1 /
// 11.9, 64 rows 12.5 / 11.9.  Partial rows of a shared prefix, 64 of them: 19.4 / 18.5.
template <bool F8>
constexpr int kNarrowRows = F8 ? 48 : 64;

template <typename T, int D, int BS, int NST, int NRAW = 0, int MODE = kPlain, int QT = 2>
__global__ void __launch_bounds__(chunk_threads<T, NRAW, MODE, QT>(), 3 - QT)
    chunk_attn_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv)
{
    using Sm = ChunkSmem<D, NST, NRAW, QT>;
    using Warps = ChunkWarps<QT>;
    constexpr int kConvThreads = 32 * Warps::kConv;
    constexpr bool kF8 = NRAW > 0;
    constexpr bool kIsMod = is_mod(MODE), kCap = has_cap(MODE), kSlope = has_slope(MODE);
    constexpr bool kBlk = is_block(MODE);
    constexpr bool kWideIO = !kCap && !kSlope;   // warps read q and write out by whole rows, but for few
    static_assert(!kBlk || kF8, "block scales belong to E4M3 caches");
    constexpr bool kTwoTerms = MODE == kPrefix;  // P as hi + lo of V's type, else one f16 term
    constexpr bool kVConv = !kF8 && std::is_same_v<T, __nv_bfloat16> && !kTwoTerms;   // bf16 V -> f16 in place
    constexpr bool kVHand = kVConv || (!kF8 && kIsMod);           // V handed over (vconv)
    constexpr bool kVZero = !kVConv && !kIsMod;    // softmax warps zero the last tile's V rows
    using TM = std::conditional_t<kF8, __half, T>;   // operand type of the score product
    constexpr int NT = kChunkTileTok;
    constexpr int BPT = NT / BS;                 // cache blocks per K/V tile
    constexpr int KS = D / 16;                   // k-steps of the score product
    constexpr bool kBf16 = DType<TM>::id == PA_BF16;
    static_assert(NT % BS == 0 && D % 64 == 0, "block_size 16/32, head_dim 64/128");

    overlap_passes<MODE>(p.num_seqs);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Sm::kBarOff);
    uint64_t* empty = full + NST;
    uint64_t* s_full = empty + NST;              // [query tile][S/P buffer]
    uint64_t* p_full = s_full + 4;               // [query tile][S/P buffer]
    uint64_t* pv_done = p_full + 4;              // [query tile]
    uint64_t* q_full = pv_done + 2;
    uint64_t* mma_done = q_full + 1;             // [query tile]
    uint64_t* v_zero = mma_done + 2;             // the last tile's V rows past the range are 0
    uint64_t* raw_full = v_zero + 1;             // [raw slot] (E4M3 caches)
    uint64_t* raw_empty = raw_full + NRAW;
    uint64_t* vconv = raw_empty + NRAW;          // [stage] (bf16 caches: V tile is f16)
    int* stage_ok = reinterpret_cast<int*>(smem + Sm::kOkOff);
    int* raw_ok = stage_ok + NST;
    float4* stage_scale = reinterpret_cast<float4*>(smem + Sm::kScaleOff);   // [stage][4] (kBlock)
    float4* raw_scale = stage_scale + NST * 4;                               // [raw slot][4]
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + Sm::kSlotOff);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // Unit (sequence, kv head, row tile) and partition of the CTA.  With modified scores the grid
    // is one-dimensional: the first p.whole_units units are one CTA each, the others are cut
    // into partitions (p.max_parts CTAs each).
    unsigned unit_y = blockIdx.y;
    int seq = blockIdx.z, part = blockIdx.x;
    bool split = MODE == kPrefix || p.partition_tokens > 0;
    if constexpr (kIsMod) {
        const int b = (int)blockIdx.x, cut = b - p.whole_units;
        const int per_seq = p.num_kv_heads * p.m_tiles;
        const int unit = cut < 0 ? b : p.whole_units + cut / p.max_parts;
        split = split && cut >= 0;
        part = split ? cut % p.max_parts : 0;
        seq = unit / per_seq;
        unit_y = unit - seq * per_seq;
    }
    const int kvh = unit_y / p.m_tiles;
    const int mt = unit_y - kvh * p.m_tiles;
    const int G = p.group;
    const int TT = p.rows_tokens;

    const int qs0 = p.query_start[seq];
    const int qs1 = p.query_start[seq + 1];
    const int n = qs1 - qs0;
    const bool rows_sane = qs0 >= 0 && n >= 0 && (int64_t)qs1 <= p.num_rows;
    // the sequence whose table row and lengths count: a group's first one (kPrefix)
    const int tseq = MODE == kPrefix ? (rows_sane && n > 0 ? qs0 : 0) : seq;
    const int L = MODE == kPrefix ? p.prefix_lens[tseq] : p.context_lens[seq];
    if (!rows_sane || L < 0 || L > p.max_context_len || n > p.max_query_len ||
        (MODE == kPrefix ? L % BS != 0 : n > L && !(takes_cross(MODE) && p.mods.all_seen))) {
        if (part == 0 && unit_y == 0 && threadIdx.x == 0)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
        if (!split && rows_sane && part == 0 && mt == 0) {
            // the sequence's rows of this kv head's query heads become NaN
            const int64_t cnt = (int64_t)n * G * D;
            for (int64_t i = threadIdx.x; i < cnt; i += blockDim.x) {
                const int64_t tok = i / ((int64_t)G * D);
                const int rem = (int)(i - tok * G * D);
                const int64_t idx = ((qs0 + tok) * p.num_q_heads + kvh * G) * D + rem;
                if (p.out_f32)
                    store_as(static_cast<float*>(p.out) + idx, __int_as_float(0x7fc00000));
                else
                    store_as(static_cast<T*>(p.out) + idx, __int_as_float(0x7fc00000));
            }
        }
        return;
    }
    if (seq == p.num_seqs - 1 && part == 0 && unit_y == 0 && threadIdx.x == 0 &&
        (int64_t)qs1 != p.num_rows)
        atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);   // rows after the last chunk belong to no one
    const int j0 = mt * TT;
    if (j0 >= n)
        return;                                  // no chunk token in this row tile
    const int ntok = min(TT, n - j0);
    const int pos_first = L - n + j0;            // position of the tile's first token
    int t_end = MODE == kPrefix ? L : pos_first + ntok;   // tokens [0, t_end) are seen by some row
    int t0 = 0, ntiles = 0;
    Seen seen{0, 0, 0};
    TileOrder order{0, 0, 0};
    int c0 = 0;                                  // kMod: first tile of the list to read
    if constexpr (kIsMod) {
        seen = seen_by(p.mods, seq, L, pos_first, pos_first + ntok - 1);
        order = seen_tiles(seen, NT);
        t_end = seen.end;
        c0 = split ? part * (p.partition_tokens / NT) : 0;
        if (c0 >= order.count) {
            // an empty context (cross attention only: a chunk's rows see themselves) gives zeros
            if (takes_cross(MODE) && order.count == 0 && !split)
                for (int i = threadIdx.x; i < ntok * G * D; i += blockDim.x) {
                    const int tok = i / (G * D);
                    const int64_t idx = ((int64_t)(qs0 + j0 + tok) * p.num_q_heads + (int64_t)kvh * G) * D +
                                        (i - tok * G * D);
                    if (p.out_f32)
                        store_as(static_cast<float*>(p.out) + idx, 0.f);
                    else
                        store_as(static_cast<T*>(p.out) + idx, 0.f);
                }
            return;
        }
        ntiles = split ? min(order.count - c0, p.partition_tokens / NT) : order.count;
    }
    int t1 = t_end;
    if constexpr (!kIsMod) {
        if (MODE == kPrefix && t_end <= 0)
            return;                              // an empty shared prefix
        if (p.partition_tokens > 0) {
            t0 = part * p.partition_tokens;
            if (t0 >= t_end)
                return;
            t1 = min(t_end, t0 + p.partition_tokens);
        }
        ntiles = (t1 - t0 + NT - 1) / NT;        // >= 1
    }
    // first token of tile it
    auto tile_token = [&](int it) -> int {
        if constexpr (kIsMod)
            return order(c0 + it) * NT;
        else
            return t0 + it * NT;
    };

    if (threadIdx.x == 0) {
#pragma unroll
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], kF8 ? Warps::kConv : 1);   // converters, or the TMA
            mbar_init(&empty[s], QT);          // one commit per issuer
        }
#pragma unroll
        for (int s = 0; s < NRAW; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], Warps::kConv);
        }
#pragma unroll
        for (int s = 0; s < NST; ++s)
            mbar_init(&vconv[s], Warps::kConv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
#pragma unroll
        for (int q = 0; q < QT; ++q) {
            mbar_init(&pv_done[q], 1);
            mbar_init(&mma_done[q], 1);
        }
        mbar_init(q_full, Warps::kSoftmax);
        mbar_init(v_zero, Warps::kSoftmax);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tslot, Sm::kTmemCols);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tslot;

    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        const int32_t* bt_row = p.block_tables + (int64_t)tseq * p.bt_stride;
        const uint64_t policy = l2_evict_first_policy();
        const int blk_end = (t1 + BS - 1) / BS;
        // 16-bit caches fill the MMA ring directly; E4M3 caches fill the raw ring
        constexpr int NP = kF8 ? NRAW : NST;
        uint64_t* pfull = kF8 ? raw_full : full;
        uint64_t* pempty = kF8 ? raw_empty : empty;
        int* pok = kF8 ? raw_ok : stage_ok;
        int issued = 0;
        // kBlock: this lane's table entry of a tile, two tiles ahead, and the scales of its block,
        // one tile ahead (loaded values are not touched before their turn: a wait for each of them,
        // tile by tile, took 1.3 us a tile)
        auto wanted = [&](int it) -> bool {
            const int b = tile_token(it) / BS + lane;
            return it < ntiles && lane < BPT && b < blk_end && any_seen(seen, b * BS, min(b * BS + BS, t1));
        };
        auto entry = [&](int it) -> int {
            return wanted(it) ? __ldg(bt_row + tile_token(it) / BS + lane) : -1;
        };
        int cur = -1, next = -1;
        RawScale sc{}, next_sc{};
        if constexpr (kBlk) {
            cur = entry(0);
            next = entry(1);
            next_sc = load_scale(p, cur, kvh);
        }
        for (int it = 0; it < ntiles; ++it) {
            const int st = it % NP;
            const int b0 = tile_token(it) / BS;
            int nb = min(BPT, blk_end - b0);
            bool want = lane < nb;
            int pbn = -1;
            bool valid = false;
            if constexpr (kBlk) {
                want = wanted(it);
                pbn = cur;
                valid = pbn >= 0 && (int64_t)pbn < p.num_blocks;
                nb = __popc(__ballot_sync(kFullMask, want));
                cur = next;
                next = entry(it + 2);
                sc = next_sc;
                next_sc = load_scale(p, cur, kvh);
            } else if constexpr (kIsMod) {        // only blocks that hold a seen token
                want = want && any_seen(seen, (b0 + lane) * BS, min((b0 + lane) * BS + BS, t1));
                nb = __popc(__ballot_sync(kFullMask, want));
            }
            if (!kBlk && want) {
                pbn = __ldg(bt_row + b0 + lane);
                valid = pbn >= 0 && (int64_t)pbn < p.num_blocks;
            }
            const unsigned vmask = __ballot_sync(kFullMask, valid);
            int ok = 1;
            if (lane == 0) {
                if (it >= NP && !mbar_wait(&pempty[st], ((it / NP) - 1) & 1)) {
                    atomicOr(p.err, PA_DEVERR_TIMEOUT);
                    ok = 0;
                } else if (!kBlk) {
                    const int nvalid = __popc(vmask);
                    pok[st] = nvalid == nb ? 1 : 0;
                    if (nvalid != nb)
                        atomicOr(p.err, PA_DEVERR_BLOCK_ID);
                    // a block is one 128-byte-row box per 64 dims (16-bit) or per 128 codes
                    mbar_arrive_expect_tx(&pfull[st],
                                          (uint32_t)nvalid * 2u * (kF8 ? 1 : Sm::kHalves) * BS * 128u);
                }
            }
            if (!__shfl_sync(kFullMask, ok, 0))
                break;
            if constexpr (kBlk) {
                // the copies go out first; the arrival follows with the scales (below)
                if (lane == 0) {
                    const int nvalid = __popc(vmask);
                    pok[st] = nvalid == nb ? 1 : 0;
                    if (nvalid != nb)
                        atomicOr(p.err, PA_DEVERR_BLOCK_ID);
                    mbar_expect_tx(&pfull[st], (uint32_t)nvalid * 2u * BS * 128u);
                }
                __syncwarp();
            }
            if (kF8 && valid) {
                unsigned char* kdst = smem + Sm::kRawOff + st * Sm::kRawStage + lane * (BS * 128);
                const int z = pbn * p.num_kv_heads + kvh;     // < 2^31 (checked on the host)
                tma_load_3d(kdst, &tk, 0, 0, z, &pfull[st], policy);
                tma_load_3d(kdst + Sm::kRawTile, &tv, 0, 0, z, &pfull[st], policy);
            } else if (valid) {
                unsigned char* kdst = smem + Sm::kStageOff + st * Sm::kStageBytes + lane * (BS * 128);
                const int z = pbn * p.num_kv_heads + kvh;     // < 2^31 (checked on the host)
#pragma unroll
                for (int h = 0; h < Sm::kHalves; ++h) {
                    tma_load_3d(kdst + h * Sm::kKVHalf, &tk, 64 * h, 0, z, &full[st], policy);
                    tma_load_3d(kdst + Sm::kKBytes + h * Sm::kKVHalf, &tv, 64 * h, 0, z, &full[st],
                                policy);
                }
            }
            if constexpr (kBlk) {
                // (scales before the copies: 1.22 us a tile, the copies waiting for them)
                if (lane < BPT)
                    raw_scale[st * 4 + lane] = block_scale(sc);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&pfull[st]);
            }
            issued = it + 1;
        }
        // no copy may still be in flight into this CTA's shared memory at exit
        if (lane == 0)
            for (int it = max(0, issued - NP); it < issued; ++it)
                mbar_wait(&pfull[it % NP], (it / NP) & 1);
        __syncwarp();
    } else if ((kF8 || kVHand) && warp >= Warps::kConv0) {
        // ------------------------------------------------ E4M3 -> f16 tile conversion
        // A raw tile row is 128 codes in 128-byte-swizzled order (16-byte chunk c of row
        // t at c ^ (t & 7)); the f16 tile is two 64-dim halves of 128-byte rows in the
        // same swizzle.  Each (token, 16-code chunk) item becomes two f16 chunks.
        if constexpr (kF8) {
            const int ct = threadIdx.x - 32 * Warps::kConv0;  // 0 .. kConvThreads - 1
            constexpr int kItems = NT * 8;                   // per K (or V) tile
            for (int it = 0; it < ntiles; ++it) {
                const int r = it % NRAW;
                const int st = it % NST;
                bool ok = mbar_wait(&raw_full[r], (it / NRAW) & 1);
                if (ok && it >= NST)
                    ok = mbar_wait(&empty[st], ((it / NST) - 1) & 1);   // both issuers' P.V
                if (!ok) {
                    if (lane == 0)
                        atomicOr(p.err, PA_DEVERR_TIMEOUT);
                    break;
                }
                const unsigned char* raw = smem + Sm::kRawOff + r * Sm::kRawStage;
                unsigned char* dst = smem + Sm::kStageOff + st * Sm::kStageBytes;
                const int tb = tile_token(it);
                const bool all_seen = !kIsMod || tile_seen(seen, tb, NT);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
#pragma unroll 4
                    for (int item = ct; item < kItems; item += kConvThreads) {
                        const int t = item >> 3;
                        const int c = item & 7;
                        uint4 w = *reinterpret_cast<const uint4*>(
                            raw + kv * Sm::kRawTile + t * 128 + ((c ^ (t & 7)) << 4));
                        if (kIsMod && kv == 1 && !all_seen && !is_seen(seen, tb + t))
                            w = make_uint4(0u, 0u, 0u, 0u);
                        unsigned char* row =
                            dst + kv * Sm::kKBytes + (c >> 2) * Sm::kKVHalf + t * 128;
                        const int c0 = 2 * (c & 3);
                        *reinterpret_cast<uint4*>(row + ((c0 ^ (t & 7)) << 4)) =
                            make_uint4(e4m3x2_to_f16x2(w.x), e4m3x2_to_f16x2(w.x >> 16),
                                       e4m3x2_to_f16x2(w.y), e4m3x2_to_f16x2(w.y >> 16));
                        *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (t & 7)) << 4)) =
                            make_uint4(e4m3x2_to_f16x2(w.z), e4m3x2_to_f16x2(w.z >> 16),
                                       e4m3x2_to_f16x2(w.w), e4m3x2_to_f16x2(w.w >> 16));
                    }
                }
                fence_proxy_async_smem();                    // f16 tiles -> tensor core
                if (kBlk && warp == Warps::kConv0 && lane < BPT)
                    stage_scale[st * 4 + lane] = raw_scale[r * 4 + lane];
                __syncwarp();
                if (lane == 0) {
                    if (warp == Warps::kConv0)
                        stage_ok[st] = raw_ok[r];
                    mbar_arrive(&full[st]);
                    mbar_arrive(&raw_empty[r]);
                }
            }
        } else if constexpr (kVConv) {
            // bf16 -> f16 of each V tile in place, once its bytes are in (the K half is
            // left to the score product meanwhile); rows past the range become 0, so
            // that 0 * V stays 0 whatever an unused slot holds.  The stage is refilled
            // only after both P.V of the tile, which wait for this hand-over.  A value
            // without an f16 value becomes infinite (or stays NaN); the epilogue reports
            // the rows it reaches.
            const int ct = threadIdx.x - 32 * Warps::kConv0;  // 0 .. kConvThreads - 1
            constexpr int kItems = NT * 8 * Sm::kHalves;     // 16-byte chunks of a V tile
            constexpr int kPer = kItems / kConvThreads;
            static_assert(kItems % kConvThreads == 0, "whole chunks per thread");
            for (int it = 0; it < ntiles; ++it) {
                const int st = it % NST;
                if (!mbar_wait(&full[st], (it / NST) & 1)) {
                    if (lane == 0)
                        atomicOr(p.err, PA_DEVERR_TIMEOUT);
                    break;
                }
                const int tb = tile_token(it);
                const int nv = min(NT, t1 - tb);              // rows inside the range
                const bool all_seen = kIsMod && tile_seen(seen, tb, NT);
                unsigned char* vt = smem + Sm::kStageOff + st * Sm::kStageBytes + Sm::kKBytes;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int item = ct + i * kConvThreads;
                    const int w = item % (NT * 8);           // chunk within a 64-dim half
                    uint4* chunk = reinterpret_cast<uint4*>(vt + (item / (NT * 8)) * Sm::kKVHalf +
                                                            w * 16);
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (kIsMod ? all_seen || is_seen(seen, tb + (w >> 3)) : (w >> 3) < nv) {
                        const uint4 b = *chunk;
                        const uint32_t in[4] = {b.x, b.y, b.z, b.w};
                        uint32_t o[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __half2 h = __floats2half2_rn(__uint_as_float(in[j] << 16),
                                                                __uint_as_float(in[j] & 0xffff0000u));
                            o[j] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        v = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    *chunk = v;
                }
                fence_proxy_async_smem();                    // f16 V -> tensor core
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&vconv[st]);
            }
        } else if constexpr (kVHand) {
            // f16 V needs no conversion: only the rows of tokens no row sees become 0
            const int ct = threadIdx.x - 32 * Warps::kConv0;
            for (int it = 0; it < ntiles; ++it) {
                const int st = it % NST;
                if (!mbar_wait(&full[st], (it / NST) & 1)) {
                    if (lane == 0)
                        atomicOr(p.err, PA_DEVERR_TIMEOUT);
                    break;
                }
                const int tb = tile_token(it);
                if (!tile_seen(seen, tb, NT)) {
                    unsigned char* vt = smem + Sm::kStageOff + st * Sm::kStageBytes + Sm::kKBytes;
                    for (int item = ct; item < NT * 8 * Sm::kHalves; item += kConvThreads) {
                        const int w = item % (NT * 8);
                        if (!is_seen(seen, tb + (w >> 3)))
                            *reinterpret_cast<uint4*>(vt + (item / (NT * 8)) * Sm::kKVHalf + w * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&vconv[st]);
            }
        }
    } else if (warp == 1 || (QT == 2 && warp == Warps::kIssuer1)) {
        // ------------------------------------------- MMA issue, one query tile per warp
        const int q = warp == 1 ? 0 : 1;
        if (lane == 0) {
            const uint32_t sq = smem_addr(smem + Sm::kQOff + q * Sm::kQTile);
            const uint32_t idesc_s = mma_idesc_f16(kBf16, kChunkRows, NT, false);
            const uint32_t idesc_o = mma_idesc_f16(kTwoTerms && kBf16, kChunkRows, D, true);   // f16 P, V
            bool ok = mbar_wait(q_full, 0);
            // S of tile it into this query tile's S buffer it & 1
            auto issue_scores = [&](int it) {
                const uint32_t kb = smem_addr(smem + Sm::kStageOff + (it % NST) * Sm::kStageBytes);
                const uint32_t dcol = tbase + Sm::kSCol + q * 128 + (it & 1) * NT;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    const uint64_t a = sw128_desc(sq + (kk / 4) * Sm::kQHalf + (kk % 4) * 32, 16, 1024);
                    const uint64_t b =
                        sw128_desc(kb + (kk / 4) * Sm::kKVHalf + (kk % 4) * 32, 16, 1024);
                    tc_mma_f16(dcol, a, b, idesc_s, kk > 0 ? 1u : 0u);
                }
                tc_commit(&s_full[q * 2 + (it & 1)]);
            };
            if (ok)
                ok = mbar_wait(&full[0], 0);
            if (ok) {
                tc_fence_after();
                issue_scores(0);
            }
            for (int it = 0; it < ntiles && ok; ++it) {
                if (it + 1 < ntiles) {
                    ok = mbar_wait(&full[(it + 1) % NST], ((it + 1) / NST) & 1);
                    // S/P buffer (it+1)&1 holds P of tile it-1 until its P.V completes
                    if (ok && it >= 1)
                        ok = mbar_wait(&pv_done[q], (it - 1) & 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    issue_scores(it + 1);
                }
                ok = mbar_wait(&p_full[q * 2 + (it & 1)], (it >> 1) & 1);
                if constexpr (kVHand) {
                    if (ok)                           // V in f16, rows past the range zeroed
                        ok = mbar_wait(&vconv[it % NST], (it / NST) & 1);
                } else if constexpr (kVZero) {
                    if (ok && t0 + (it + 1) * NT > t1)
                        ok = mbar_wait(v_zero, 0);   // last tile: V rows past the range zeroed
                }
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t vb =
                    smem_addr(smem + Sm::kStageOff + (it % NST) * Sm::kStageBytes + Sm::kKBytes);
                const uint32_t pcol = tbase + Sm::kSCol + q * 128 + (it & 1) * NT;
#pragma unroll
                for (int kk = 0; kk < NT / 16; ++kk) {        // 16 tokens = 8 columns of P
                    const uint64_t b = sw128_desc(vb + kk * 16 * 128, Sm::kKVHalf, 1024);
                    tc_mma_f16_ts(tbase + q * 128, pcol + kk * 8, b, idesc_o,
                                  (it > 0 || kk > 0) ? 1u : 0u);
                    if constexpr (kTwoTerms)
                        tc_mma_f16_ts(tbase + q * 128, pcol + NT / 2 + kk * 8, b, idesc_o, 1u);
                }
                tc_commit(&pv_done[q]);
                tc_commit(&empty[it % NST]);
            }
            if (!ok)
                atomicOr(p.err, PA_DEVERR_TIMEOUT);
            tc_commit(&mma_done[q]);          // every MMA above completes before TMEM is freed
            mbar_wait(&mma_done[q], 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax warps
        const int q = (warp - 2) >> 2;                   // query tile of this warp
        const int wq = warp & 3;                         // TMEM lane quarter of this warp
        const int rr = 32 * wq + lane;                   // row within the query tile = TMEM lane
        const int r = q * kChunkRows + rr;               // row within the CTA
        const int tok = r / G;
        const int g = r - tok * G;
        const bool row_valid = tok < ntok;               // (r >= TT * G gives tok >= TT)
        const int pos = MODE == kPrefix ? L - 1 : pos_first + tok;
        // kMod: first visible position past the global tokens, base-2 distance slope
        const int low = kIsMod && p.mods.window > 0 ? max(0, pos - p.mods.window + 1) : 0;
        const float slope = kSlope ? base2_slope(p.mods.slopes[kvh * G + g]) : 0.f;
        const int64_t qrow = (int64_t)(qs0 + j0 + tok) * p.num_q_heads + (int64_t)kvh * G + g;
        // scores are used as s * sl2 with sl2 > 0: a negative scale flips the sign of q
        // (exact), a zero scale makes q zero (every score 0); over E4M3 caches the K scale
        // of the kv head joins the softmax scale (kBlock: the one of a block, tile by tile)
        const float sl2_raw = kF8 && !kBlk ? p.scale_log2 * p.k_scale[kvh] : p.scale_log2;
        const uint32_t qflip = sl2_raw < 0.f ? 0x80008000u : 0u;
        const bool qzero = sl2_raw == 0.f;
        float sl2 = qzero ? 1.f : fabsf(sl2_raw);
        // kWideIO: a row is CPR lanes of 16 bytes wide; rows of q and out (all heads) from the CTA's
        // first one, -1: none
        constexpr int CPR = D / 8, RPW = 32 / CPR;
        const int64_t row_base = (int64_t)(qs0 + j0) * p.num_q_heads + (int64_t)kvh * G;
        const int my_row = row_valid ? tok * p.num_q_heads + g : -1;
        const bool wide = kWideIO && (MODE == kPrefix || ntok * G > kNarrowRows<kF8>);
        {
            // Q rows into the 128-byte-swizzled operand layout; rows past the chunk are 0.  The
            // lanes of a warp read whole rows (CPR lanes of 16 bytes each), not one row a lane:
            // with the epilogue's stores, which go the same way, one row a lane cost a CTA of 256 rows
            // 2 to 5 us at head_dim 128 (over 64 tokens 12.2 against 10.1 us; 4 x 512 tokens of 8192,
            // 64/8 heads, bf16, 526 against 511).  At head_dim 64 few rows are read a row a lane, as
            // they are written (kNarrowRows; 40 rows under a window of 128, 7.5 against 7.0 us).
            // Capped and biased scores keep a row a lane: their loops lose more to the registers
            // (568 against 608 us, capped, f16).
            if (kWideIO && (D == 128 || wide)) {
                unsigned char* qdst = smem + Sm::kQOff + q * Sm::kQTile + 32 * wq * 128;
                constexpr bool kToF16 = kF8 && DType<T>::id == PA_BF16;
                const uint4* src =
                    reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + row_base * D) + lane % CPR;
                uint4 qv[CPR];
#pragma unroll
                for (int i = 0; i < CPR; ++i) {
                    const int row = __shfl_sync(kFullMask, qzero ? -1 : my_row, i * RPW + lane / CPR);
                    qv[i] = row >= 0 ? __ldg(src + (int64_t)row * CPR) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < CPR; ++i) {
                    const int r32 = i * RPW + lane / CPR, c = lane % CPR;
                    if constexpr (kToF16) {
                        // a bf16 row becomes f16 operands: a power of two 2^-e puts its largest
                        // |q| in [2^14, 2^15), so the 8-bit mantissas convert exactly; 2^e goes
                        // into the row's score scale
                        uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
                        float amax = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)),
                                                     fabsf(__uint_as_float(w[j] & 0xffff0000u))));
                        // over the lanes of either row (magnitudes order as their bits do)
                        static_assert(!kToF16 || RPW == 2, "two rows a step");
                        const unsigned bits = __float_as_uint(amax);
                        const unsigned lo = __reduce_max_sync(kFullMask, lane < 16 ? bits : 0u);
                        const unsigned hi = __reduce_max_sync(kFullMask, lane < 16 ? 0u : bits);
                        amax = __uint_as_float(lane < 16 ? lo : hi);
                        const int ex = (__float_as_int(amax) >> 23) & 0xff;   // biased exponent
                        // amax in [2^(ex-127), 2^(ex-126)): scale by 2^(141 - ex); rows of zeros,
                        // tiny rows and a NaN / infinite row keep the scale 1
                        const int sh = (ex == 0 || ex == 255) ? 0 : max(-100, min(100, 141 - ex));
                        const float down = __int_as_float((127 + sh) << 23);
                        const int own = __shfl_sync(kFullMask, sh, lane % RPW * CPR);   // of row i RPW + lane % RPW
                        if (lane / RPW == i)
                            sl2 *= __int_as_float((127 - own) << 23);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __half2 h = __floats2half2_rn(__uint_as_float(w[j] << 16) * down,
                                                                __uint_as_float(w[j] & 0xffff0000u) * down);
                            w[j] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        qv[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    qv[i].x ^= qflip;
                    qv[i].y ^= qflip;
                    qv[i].z ^= qflip;
                    qv[i].w ^= qflip;
                    *reinterpret_cast<uint4*>(qdst + (c / 8) * Sm::kQHalf + r32 * 128 + (((c & 7) ^ (r32 & 7)) << 4)) =
                        qv[i];
                }
            } else {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                                  (row_valid ? qrow : 0) * D);
                unsigned char* qdst = smem + Sm::kQOff + q * Sm::kQTile + rr * 128;
                constexpr bool kToF16 = kF8 && DType<T>::id == PA_BF16;
                float down = 1.f;
                if constexpr (kToF16) {
                    // a bf16 row becomes f16 operands: a power of two 2^-e puts its largest
                    // |q| in [2^14, 2^15), so the 8-bit mantissas convert exactly; 2^e goes
                    // into the row's score scale
                    float amax = 0.f;
                    if (row_valid && !qzero) {
#pragma unroll 4
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 v = __ldg(src + c);
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)),
                                                         fabsf(__uint_as_float(w[j] & 0xffff0000u))));
                        }
                    }
                    const int ex = (__float_as_int(amax) >> 23) & 0xff;   // biased exponent
                    // amax in [2^(ex-127), 2^(ex-126)): scale by 2^(141 - ex); rows of zeros,
                    // tiny rows and a NaN / infinite row keep the scale 1
                    const int sh = (ex == 0 || ex == 255) ? 0 : max(-100, min(100, 141 - ex));
                    down = __int_as_float((127 + sh) << 23);
                    sl2 *= __int_as_float((127 - sh) << 23);
                }
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (row_valid && !qzero) {
                        v = __ldg(src + c);
                        if constexpr (kToF16) {
                            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __half2 h = __floats2half2_rn(__uint_as_float(w[j] << 16) * down,
                                                                    __uint_as_float(w[j] & 0xffff0000u) * down);
                                w[j] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            v = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        v.x ^= qflip;
                        v.y ^= qflip;
                        v.z ^= qflip;
                        v.w ^= qflip;
                    }
                    *reinterpret_cast<uint4*>(qdst + (c / 8) * Sm::kQHalf + (((c & 7) ^ (rr & 7)) << 4)) = v;
                }
            }
        }
        if constexpr (kF8 && !kBlk)
            sl2 = score_factor(sl2);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(q_full);

        // Capped scores, fast form: for |y| <= kCapNear, y = s kk, tanh y = y P(y^2) (see
        // cap_score_near), so the score is s (kp0 + kp1 s^2 + kp2 s^4 + kp3 s^6): three packed
        // multiply-adds more than an uncapped score, and no MUFU work beyond its one exp2.
        // Taken by a warp's tile that all its rows see whole and whose scores lie in that
        // range; other tiles take cap_row.  With kk in [10^-6, 8] the powers of kk and, as
        // |s| <= 0.5 / kk, of s are normal numbers.  kp3 may be subnormal or 0 where sl2 is tiny as
        // well; its term then errs by at most 2^-150 |s|^7 <= 6 10^-48 / kk^7, 6 10^-6 of a score
        // in base-2 units.
        // Over E4M3 caches, where bf16 rows came in as 2^e q and kk is as small, the polynomial is
        // of y itself, one multiply more (always cap_score: 798 against 628 us, 4 x 512 tokens of 8192).
        const float kk = kCap ? sl2 * p.mods.inv_cap : 0.f;
        const bool cap_fast = kCap && !kSlope && __all_sync(kFullMask, kF8 || (kk >= 1e-6f && kk <= 8.f));
        const float k1 = kF8 ? p.mods.cap : sl2, k2 = kF8 ? 1.f : kk * kk;
        const float kp[4] = {kCapP0 * k1, kCapP1 * k1 * k2, kCapP2 * k1 * k2 * k2,
                             kCapP3 * k1 * k2 * k2 * k2};
        auto poly_at = [&](float z) { return fmaf(fmaf(fmaf(kp[3], z, kp[2]), z, kp[1]), z, kp[0]); };
        const bool warp_live = __any_sync(kFullMask, row_valid);
        const uint32_t lane_t = tbase + ((uint32_t)(32 * wq) << 16);
        const uint32_t o_col = lane_t + q * 128;
        float m_ref = -INFINITY, lsum = 0.f;
        bool poisoned = false;
        for (int it = 0; it < ntiles; ++it) {
            const int b = it & 1;
            const int st = it % NST;
            const int tb = tile_token(it);
            bool ok = mbar_wait(&s_full[q * 2 + b], (it >> 1) & 1);
            ok = ok && mbar_wait(&full[st], (it / NST) & 1);   // stage_ok and the tile's bytes
            if (!ok) {
                if (lane == 0)
                    atomicOr(p.err, PA_DEVERR_TIMEOUT);
                poisoned = true;
                break;
            }
            if (!stage_ok[st])
                poisoned = true;
            tc_fence_after();
            const uint32_t sp_col = lane_t + Sm::kSCol + q * 128 + b * NT;   // this row's S/P buffer
            float s[NT];
            if (warp_live)
                tmem_ld64(sp_col, s);
            if (warp_live) {
                const int lim = row_valid ? pos - tb : -1;   // columns c <= lim are visible
                float mul = sl2;                 // scores are s * mul (base 2), or, capped, the
                bool poly = false;               // polynomial of s below
                float smax;
                if constexpr (kIsMod) {
                    // column c is visible when c < gl, or lo <= c <= lim (rows past the
                    // chunk are all zeros and never stored: let them see everything)
                    const int gl = seen.glob - tb, lo = low - tb;
                    const bool whole = __all_sync(
                        kFullMask, !row_valid || gl >= NT || (lim >= NT - 1 && lo <= 0));
                    if constexpr (kCap && !kSlope) {
                        if (whole && cap_fast) {
                            const float2 mm = row_range(s);
                            smax = mm.y;
                            poly = __all_sync(kFullMask, fmaxf(fabsf(mm.x), fabsf(mm.y)) * kk <= kCapNear);
                        }
                    }
                    if (!poly) {
                        if constexpr (kCap) {
                            mul = 1.f;
                            cap_row(s, sl2, p.mods, whole);
                        }
                        if constexpr (kSlope) {
                            // |pos - t| = pos - t while no column lies behind pos
                            const float far0 = (float)(pos - tb);
                            if (lim >= NT - 1 || !row_valid) {
                                // the bias of columns c, c + 1 advances by eight columns at a time
                                // (eight roundings a tile at most)
                                const float2 one = make_float2(1.f, 1.f);
                                const float2 step = make_float2(8.f * slope, 8.f * slope);
                                float2 d[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    d[k] = make_float2(-slope * (far0 - (float)(2 * k)),
                                                       -slope * (far0 - (float)(2 * k + 1)));
#pragma unroll
                                for (int c = 0; c < NT; c += 2) {
                                    const int k = (c >> 1) & 3;
                                    const float2 x = ffma2(make_float2(s[c], s[c + 1]),
                                                           make_float2(mul, mul), d[k]);
                                    d[k] = ffma2(step, one, d[k]);
                                    s[c] = x.x;
                                    s[c + 1] = x.y;
                                }
                            } else {
#pragma unroll
                                for (int c = 0; c < NT; ++c)
                                    s[c] = fmaf(-slope, fabsf(far0 - (float)c), s[c] * mul);
                            }
                            mul = 1.f;
                        }
                        if (!whole) {
                            // bits of the visible columns (a row past the chunk: all)
                            auto below = [](int n) -> uint64_t {      // bits 0 .. n - 1
                                return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
                            };
                            const uint64_t vis = row_valid ? below(gl) | (below(lim + 1) & ~below(lo)) : ~0ull;
#pragma unroll
                            for (int c = 0; c < NT; ++c)
                                s[c] = (vis >> c) & 1ull ? s[c] : -INFINITY;
                        }
                        if constexpr (!kBlk)
                            smax = row_max(s);
                    }
                } else {
                    if (lim < NT - 1) {
#pragma unroll
                        for (int c = 0; c < NT; ++c)
                            s[c] = c <= lim ? s[c] : -INFINITY;
                    }
                    smax = row_max(s);
                }
                float tmax;
                if constexpr (kBlk) {
                    tmax = -INFINITY;
#pragma unroll
                    for (int k = 0; k < BPT; ++k) {
                        float mx[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mx[i] = max3f(s[k * BS + i], s[k * BS + 4 + i], s[k * BS + 8 + i]);
#pragma unroll
                        for (int c = 12; c + 8 <= BS; c += 8)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mx[i] = max3f(mx[i], s[k * BS + c + i], s[k * BS + c + 4 + i]);
                        const float top = max3f(s[k * BS + BS - 4], s[k * BS + BS - 3],
                                                fmaxf(s[k * BS + BS - 2], s[k * BS + BS - 1]));
                        const float4 sc = stage_scale[st * 4 + k];
                        tmax = fmaxf(tmax, fmaf(max3f(max3f(mx[0], mx[1], mx[2]), mx[3], top), score_factor(sl2 * sc.x),
                                                sc.y));
                    }
                } else {
                    tmax = smax == -INFINITY ? -INFINITY : smax * mul;
                }
                if (kCap && poly) {
                    const float y = kF8 ? smax * kk : smax;
                    tmax = y * poly_at(y * y);
                }
                const bool need = tmax > m_ref + 8.f;
                if (it > 0 && __any_sync(kFullMask, need)) {
                    // O holds P.V of tiles 0 .. it-1: wait for the last, then rescale the
                    // rows whose reference maximum moves
                    if (!mbar_wait(&pv_done[q], (it - 1) & 1)) {
                        if (lane == 0)
                            atomicOr(p.err, PA_DEVERR_TIMEOUT);
                        poisoned = true;
                    }
                    tc_fence_after();
                    const float alpha = need ? ex2_approx(m_ref - tmax) : 1.f;
#pragma unroll 1
                    for (int c4 = 0; c4 < D / 32; ++c4) {
                        float o[32];
                        tmem_ld32(o_col + 32 * c4, o);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 v = fmul2(make_float2(o[i], o[i + 1]), make_float2(alpha, alpha));
                            o[i] = v.x;
                            o[i + 1] = v.y;
                        }
                        tmem_st32(o_col + 32 * c4, o);
                    }
                }
                if (need) {
                    lsum *= ex2_approx(m_ref - tmax);
                    m_ref = tmax;
                }
                // 2^7 p = 2^(s * sl2 - m_ref + 7), in place; 0 where masked (s = -inf) or no
                // reference; the row sum carries the same 2^7
                const float nm = (m_ref == -INFINITY ? 0.f : -m_ref) + kChunkPExp;
                float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                 make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                if constexpr (kBlk) {
                    // w = 2^7 2^(s sl2 s_k + log2 u_k - m_ref), the sum of w / u_k (block_scale.cuh)
#pragma unroll
                    for (int k = 0; k < BPT; ++k) {
                        const float4 sc = stage_scale[st * 4 + k];
                        const float mul_k = score_factor(sl2 * sc.x);
                        const float2 f = make_float2(mul_k, mul_k), add = make_float2(nm + sc.y, nm + sc.y);
                        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int c = k * BS; c < (k + 1) * BS; c += 2) {
                            const float2 x = ffma2(make_float2(s[c], s[c + 1]), f, add);
                            s[c] = ex2_approx(x.x);
                            s[c + 1] = ex2_approx(x.y);
                            part[(c >> 1) & 1] = ffma2(make_float2(s[c], s[c + 1]), make_float2(1.f, 1.f),
                                                       part[(c >> 1) & 1]);
                        }
                        lsum = fmaf((part[0].x + part[0].y) + (part[1].x + part[1].y), sc.z, lsum);
                    }
                }
                // (one loop for either form of the scores: a test in one loop for both cost 13 %
                // where the cap bites)
                auto weights = [&](auto capped) {
#pragma unroll
                    for (int c = 0; c < NT; c += 2) {
                        float2 f = make_float2(mul, mul), y = make_float2(s[c], s[c + 1]);
                        if constexpr (capped.value) {
                            if (kF8)
                                y = fmul2(y, make_float2(kk, kk));
                            const float2 z = fmul2(y, y);
                            f = ffma2(z, make_float2(kp[3], kp[3]), make_float2(kp[2], kp[2]));
                            f = ffma2(z, f, make_float2(kp[1], kp[1]));
                            f = ffma2(z, f, make_float2(kp[0], kp[0]));
                        }
                        const float2 x = ffma2(y, f, make_float2(nm, nm));
                        s[c] = ex2_approx(x.x);
                        s[c + 1] = ex2_approx(x.y);
                        acc[(c >> 1) & 3] = ffma2(make_float2(s[c], s[c + 1]), make_float2(1.f, 1.f),
                                                  acc[(c >> 1) & 3]);
                    }
                };
                if constexpr (kCap && !kSlope) {
                    if (poly)
                        weights(std::true_type{});
                    else
                        weights(std::false_type{});
                } else if constexpr (!kBlk) {
                    weights(std::false_type{});
                }
                if constexpr (!kBlk)
                    lsum += ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) +
                        ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y));
            }
            if (kTwoTerms && warp_live) {
                // P over the S buffer: hi pairs in the first 32 columns, lo pairs in the others
                uint32_t w[NT];
#pragma unroll
                for (int k = 0; k < NT / 2; ++k) {
                    w[k] = pack_pair<TM>(s[2 * k], s[2 * k + 1]);
                    const float2 f = unpack_pair<TM>(w[k]);
                    const float2 d = ffma2(f, make_float2(-1.f, -1.f), make_float2(s[2 * k], s[2 * k + 1]));
                    w[NT / 2 + k] = pack_pair<TM>(d.x, d.y);
                }
                tmem_st64_raw(sp_col, w);
            } else if (warp_live) {
                // P over the first 32 columns of the S buffer, as f16 pairs
                uint32_t ph[NT / 2];
#pragma unroll
                for (int k = 0; k < NT / 2; ++k) {
                    const __half2 h = __floats2half2_rn(s[2 * k], s[2 * k + 1]);
                    ph[k] = *reinterpret_cast<const uint32_t*>(&h);
                }
                tmem_st32_raw(sp_col, ph);
            }
            if (kVZero && tb + NT > t1) {
                // V rows past the range may hold anything (unused slots, stale tiles):
                // zero them so that 0 * V stays 0; both issuers wait for v_zero before
                // their last P.V
                const int v0 = t1 - tb;
                const int rows = NT - v0;
                unsigned char* vbase = smem + Sm::kStageOff + st * Sm::kStageBytes + Sm::kKBytes;
                for (int idx = threadIdx.x - 64; idx < Sm::kHalves * rows * 8;
                     idx += 32 * Warps::kSoftmax) {
                    const int h = idx / (rows * 8);
                    const int w = idx - h * rows * 8;
                    *reinterpret_cast<uint4*>(vbase + h * Sm::kKVHalf + (v0 + w / 8) * 128 +
                                              (w % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(v_zero);
            }
            tc_fence_before();                           // the P store precedes P.V
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&p_full[q * 2 + b]);
        }

        // ---------------------------------------------------------------- epilogue
        // every MMA of this query tile has completed once its issuer's final commit has
        // (one phase, so no parity wait can alias: P.V of the last two tiles may be pending
        // or done in any combination when a warp gets here)
        if (!mbar_wait(&mma_done[q], 0)) {
            if (lane == 0)
                atomicOr(p.err, PA_DEVERR_TIMEOUT);
            poisoned = true;
        }
        tc_fence_after();
        if (warp_live) {
            // over E4M3 caches the V scale of the kv head multiplies the output
            const float inv = lsum > 0.f ? (kF8 && !kBlk ? p.v_scale[kvh] : 1.f) / lsum : 0.f;
            const int which = (split || p.out_f32) ? 0 : (DType<T>::id == PA_F16 ? 1 : 2);
            // over a bf16 cache, O that is not finite while the probabilities and their
            // sum are means the row weighed a V element without an f16 value (O itself
            // cannot overflow: |O| <= l max|v|, far inside fp32)
            const bool watch = kVConv && row_valid && !poisoned && lsum > 0.f && lsum < INFINITY;
            bool unconvertible = false;
            if (wide) {
                // Rows go out through this warp's 32 rows of the query tile (no product reads them any
                // more), so that its lanes store whole rows; piece c of a row at c ^ (row & 7).
                unsigned char* stage = smem + Sm::kQOff + q * Sm::kQTile + 32 * wq * 128;
                auto piece = [&](int r32, int c) -> uint4* {
                    return reinterpret_cast<uint4*>(stage + (c / 8) * Sm::kQHalf + r32 * 128 +
                                                    (((c & 7) ^ (r32 & 7)) << 4));
                };
#pragma unroll 1
                for (int c4 = 0; c4 < D / 32; ++c4) {
                    float o[32];
                    tmem_ld32(o_col + 32 * c4, o);
                    if (watch)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            unconvertible |= !(fabsf(o[i]) < INFINITY);
                    if (which != 0) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *piece(lane, 4 * c4 + k) = pack_out8(o + 8 * k, inv, poisoned, which);
                        continue;
                    }
                    // fp32: 32 columns are 128 bytes of a row
                    const float qnan = __int_as_float(0x7fc00000);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 f = poisoned ? make_float4(qnan, qnan, qnan, qnan)
                                                  : make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv,
                                                                o[4 * k + 3] * inv);
                        *piece(lane, k) = *reinterpret_cast<const uint4*>(&f);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = __shfl_sync(kFullMask, my_row, 4 * i + lane / 8);
                        if (row >= 0) {
                            float* dst = split ? p.part_o + ((row_base + row) * p.max_parts + part) * D
                                               : static_cast<float*>(p.out) + (row_base + row) * D;
                            *reinterpret_cast<uint4*>(dst + 32 * c4 + 4 * (lane % 8)) = *piece(4 * i + lane / 8, lane % 8);
                        }
                    }
                    __syncwarp();
                }
                if (which != 0) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < CPR; ++i) {
                        const int r32 = i * RPW + lane / CPR;
                        const int row = __shfl_sync(kFullMask, my_row, r32);
                        if (row >= 0)
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (row_base + row) * D +
                                                      8 * (lane % CPR)) = *piece(r32, lane % CPR);
                    }
                }
                if (split && row_valid) {
                    const int64_t prw = qrow * p.max_parts + part;
                    p.part_ml[prw * 2 + 0] = poisoned ? __int_as_float(0x7fc00000) : m_ref;
                    // the sum carries 2^7; the suffix rows it is merged with do not
                    p.part_ml[prw * 2 + 1] = MODE == kPrefix ? lsum * 0x1p-7f : lsum;
                }
            } else {
#pragma unroll 1
                for (int c4 = 0; c4 < D / 32; ++c4) {
                    float o[32];
                    tmem_ld32(o_col + 32 * c4, o);
                    if (!row_valid)
                        continue;
                    if (watch)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            unconvertible |= !(fabsf(o[i]) < INFINITY);
                    if (split) {
                        const int64_t prw = qrow * p.max_parts + part;
                        store_row32(p.part_o, prw * D + 32 * c4, o, inv, poisoned, 0);
                        if (c4 == 0) {
                            p.part_ml[prw * 2 + 0] = poisoned ? __int_as_float(0x7fc00000) : m_ref;
                            // the sum carries 2^7; the suffix rows it is merged with do not
                            p.part_ml[prw * 2 + 1] = MODE == kPrefix ? lsum * 0x1p-7f : lsum;
                        }
                    } else {
                        store_row32(p.out, qrow * D + 32 * c4, o, inv, poisoned, which);
                    }
                }
            }
            if (kVConv && __any_sync(kFullMask, unconvertible) && lane == 0)
                atomicOr(p.err, PA_DEVERR_RANGE);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, Sm::kTmemCols);
    }
}

// Merges the partitions of a split chunk launch: one CTA of D threads per
// (query row, query head); grid = (rows, num_q_heads).
template <typename T, int D>
__global__ void __launch_bounds__(D) chunk_reduce_kernel(const ChunkParams p)
{
    const int64_t row = blockIdx.x;
    const int h = blockIdx.y;
    const int d = threadIdx.x;
    // the sequence owning the row: query_start[s] <= row < query_start[s + 1]
    int lo = 0, hi = p.num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.query_start[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    const int s = lo;
    const int qs0 = p.query_start[s], qs1 = p.query_start[s + 1];
    const int n = qs1 - qs0;
    const int L = p.context_lens[s];
    const int64_t idx = (row * p.num_q_heads + h) * D + d;
    float out;
    if (row < qs0 || row >= qs1 || n > L || L < 0 || L > p.max_context_len || n > p.max_query_len) {
        out = __int_as_float(0x7fc00000);
        if (d == 0 && h == 0)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
    } else {
        const int pos = L - n + (int)(row - qs0);
        const int nparts = min(p.max_parts, (pos + p.partition_tokens) / p.partition_tokens);
        const int64_t prow0 = (row * p.num_q_heads + h) * p.max_parts;
        float M = -INFINITY;
        for (int k = 0; k < nparts; ++k)
            M = fmaxf(M, p.part_ml[(prow0 + k) * 2]);
        float num = 0.f, den = 0.f;
        for (int k = 0; k < nparts; ++k) {
            const float mk = p.part_ml[(prow0 + k) * 2];
            const float w = mk == -INFINITY ? 0.f : exp2f(mk - M) * p.part_ml[(prow0 + k) * 2 + 1];
            num = fmaf(w, p.part_o[(prow0 + k) * D + d], num);
            den += w;
        }
        // a poisoned partition (NaN) makes the row NaN; no visible token gives 0
        out = den > 0.f ? num / den : (den == 0.f ? 0.f : __int_as_float(0x7fc00000));
    }
    if (p.out_f32)
        store_as(static_cast<float*>(p.out) + idx, out);
    else
        store_as(static_cast<T*>(p.out) + idx, out);
}

}  // namespace pa
