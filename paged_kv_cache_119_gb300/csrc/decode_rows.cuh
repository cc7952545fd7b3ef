// decode_rows.cuh -- paged attention of 9 to 64 rows of a kv head on mma.sync (sm_103a): the
// (token, head) rows of a short chunk, the heads of a wide group, or the (sequence, head) rows
// of a group that shares a prefix; fp16 / bf16 caches, and E4M3 caches at head_dim 128, or with
// block scales at 64 too.
//
// decode_mma_kernel puts 16 tokens on the M side of the matrix instruction and 8 rows on the
// N side, which suits 8 rows: their K and V fragments feed nothing else.  With more rows that
// form repeats every K and V fragment load and the whole softmax bookkeeping per 8 rows, and
// measured about 6.4 (16 tokens x 8 rows) steps a microsecond per SM whatever the memory does.
// Here 16 rows are the M side:
//   S[16 rows x 8 tok] = Q . K^T     A = Q fragments in registers, B = K by ldmatrix
//   O[16 rows x 8 dims] += P . V     A = P straight from the accumulators of S (its layout is
//                                    the A layout), B = V by ldmatrix.trans
// so a K or V fragment feeds 16 rows, nothing is transposed in registers, and a row's maximum
// takes two shuffles.  P enters as hi + lo halves of the 16-bit type (2^-16 relative), sums and
// maxima are fp32, as in decode_mma_kernel.
//
// Organisation: a producer warp and four consumer warps around a ring of TMA tiles, as in
// decode_mma_kernel.  A CTA serves RW row groups of 16 rows; consumer warp w takes row group
// w % RW of the tiles w / RW, w / RW + 4 / RW, .., so RW warps share a tile, and up to 64 rows
// share one read of K and V.  The warps of a row group merge through shared memory at the end.
// Bound: HBM where 16 rows or fewer share a byte, issue slots of mma.sync and softmax beyond.
// 32 sequences of 5 new tokens, 4 heads a kv head, f16, a window of 1024: 33.7 us (4.1 TB/s);
// the pass over 16 prefixes of 1024 tokens for 8 x 4 rows each, bf16: 18 us.  On decode_mma_kernel
// (8 rows a CTA) the first took 89 us, on a transposed tcgen05 form of 16 and 32 rows 65.
// Modes: kMod and kBlock (chunk rows, or with query_start null the heads of each sequence's last token;
// kModBoth when the scores have a cap or slopes),
// kPrefix and kSuffix, which write partial rows only.
#pragma once

#include "decode_mma.cuh"

namespace pa {

constexpr int kRowsGroup = 16;       // rows of a consumer warp
constexpr int kRowsTile = 32;        // tokens of a K/V tile

template <typename TK, int D, int NSTAGE, int RW>
struct RowsSmem {
    static constexpr int TB = kRowsTile;
    static constexpr bool kFp8 = sizeof(TK) == 1;
    static constexpr int kTileBytes = TB * D * (int)sizeof(TK);          // one K (or V) tile
    static constexpr int kHalfBytes = TB * 128;                          // one 128-byte-row box
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRingBytes = NSTAGE * kStageBytes;
    // merge area (over the ring, once every tile is consumed): 16 rows of each warp, D + 8
    // floats apart so that the 8-byte stores of a fragment meet no bank twice
    static constexpr int kMergeRow = D + 8;
    static constexpr int kMergeAcc = kDecodeConsumerWarps * kRowsGroup * kMergeRow * 4;
    static constexpr int kMergeBytes = kMergeAcc + kDecodeConsumerWarps * kRowsGroup * 2 * 4;
    static constexpr int kDataBytes = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static constexpr int kBarOffset = (kDataBytes + 7) / 8 * 8;
    static constexpr int kOkOffset = kBarOffset + 2 * NSTAGE * 8;
    static constexpr int kFlagOffset = kOkOffset + NSTAGE * 4;
    static constexpr int kBytes = kFlagOffset + 16;
    static constexpr int kAlloc = kBytes + 1024;                         // room to align to 1 KB
    // kBlock: the scales of the CTA's blocks behind all that
    static constexpr int kScaleOffset = (kBytes + 15) / 16 * 16;
    static constexpr int kAllocBlock = kScaleOffset + kScaleRingBytes + 1024;
    static_assert(kHalfBytes % 1024 == 0, "swizzle atoms need 1 KB alignment");
};

// CTAs per SM.  The small tiles of kBlock at head_dim 64 want warps (16 x 8192 tokens, 128/8 heads,
// blocks of 16: 65.7 us with two, 52.0 with three, 45.7 with four; 64 rows a CTA: 130, 131, 136).
template <int D, int MODE, int RW>
constexpr int rows_min_blocks() { return D == 64 && is_block(MODE) ? (RW == 4 ? 3 : 4) : 2; }

// T: query / native output type.  TK: T, or __nv_fp8_e4m3 (value = code * per-kv-head scale).
// A tile is 32 tokens: one cache block, or two of 16.
template <typename T, typename TK, int D, int BS, int NSTAGE, int MODE, int RW>
__global__ void __launch_bounds__(kDecodeThreads, rows_min_blocks<D, MODE, RW>())
    decode_rows_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv)
{
    constexpr int TB = kRowsTile;
    constexpr int BPT = TB / BS;
    using Sm = RowsSmem<TK, D, NSTAGE, RW>;
    constexpr bool kFp8 = Sm::kFp8;
    using TM = std::conditional_t<kFp8, __half, T>;   // matrix operand type
    constexpr int NCW = kDecodeConsumerWarps;
    constexpr int TW = NCW / RW;      // warps that share out the tiles of a row group
    constexpr int NR = kRowsGroup * RW;
    constexpr int KS = D / 16;        // k-steps of the score product
    constexpr int NB = D / 8;         // 8-dim column blocks of O
    constexpr bool kIsMod = is_mod(MODE), kBlk = is_block(MODE);
    static_assert(!kFp8 || D == 128 || kBlk, "E4M3 tiles are read in place: head_dim 128, or kBlock's maps");
    static_assert(!kBlk || (kFp8 && NSTAGE * BPT <= 32), "the ring of scales outlasts the ring of tiles");
    static_assert(kIsMod || MODE == kPrefix || MODE == kSuffix, "the plain mode has its own kernels");
    static_assert(NCW % RW == 0 && NSTAGE % NCW == 0, "each ring stage belongs to one warp of a row group");
    static_assert((BS == 16 || BS == 32) && D % 64 == 0, "block_size 16/32, head_dim 64/128");

    if (overlap_passes<MODE>(p.num_seqs))
        return;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Sm::kBarOffset);
    uint64_t* empty = full + NSTAGE;
    int* stage_ok = reinterpret_cast<int*>(smem + Sm::kOkOffset);
    int* poison = reinterpret_cast<int*>(smem + Sm::kFlagOffset);
    float4* scales = reinterpret_cast<float4*>(smem + Sm::kScaleOffset);    // kBlock

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int seq = blockIdx.z;
    const int kvh = blockIdx.y / p.chunks;
    const int R0 = (blockIdx.y - kvh * p.chunks) * NR;   // the CTA's first row of the kv head
    const int part = blockIdx.x;
    const bool split = MODE == kPrefix || MODE == kSuffix || p.partition_tokens > 0;

    // the sequence's (or group's) rows of q / out are qs0 .. qs0 + n - 1
    int qs0 = seq, n = 1;
    if (MODE == kPrefix || (kIsMod && p.query_start)) {
        qs0 = p.query_start[seq];
        n = p.query_start[seq + 1] - qs0;
    }
    const bool rows_sane = qs0 >= 0 && n >= 0 && (int64_t)qs0 + n <= p.num_rows;
    // the sequence whose table row and lengths count: a group's first one (kPrefix)
    const int tseq = MODE == kPrefix ? (rows_sane && n > 0 ? qs0 : 0) : seq;
    int L, start = 0;                             // the tokens of this pass are start .. L - 1
    bool bad_len;
    if constexpr (MODE == kPrefix) {
        L = p.prefix_lens[tseq];
        bad_len = L < 0 || L > p.max_prefix_len || L % BS != 0 || n > p.max_query_len;
    } else {
        L = p.context_lens[seq];
        bad_len = L < 0 || L > p.max_context_len;
        if constexpr (MODE == kSuffix) {
            start = p.prefix_lens[seq];
            bad_len = bad_len || start < 0 || start > p.max_prefix_len || start % BS != 0 || start > L ||
                      L - start > p.max_suffix_len;
        } else if (p.query_start) {
            bad_len = bad_len || (n > L && !(takes_cross(MODE) && p.mods.all_seen)) || n > p.max_query_len;
        }
    }
    // the q / out row of row R of the kv head (R / group < n)
    auto out_row = [&](int R) -> int64_t {
        const int j = R / p.group;
        return (int64_t)(qs0 + j) * p.num_q_heads + (int64_t)kvh * p.group + (R - j * p.group);
    };
    if (bad_len || !rows_sane) {
        if (part == 0 && blockIdx.y == 0 && threadIdx.x == 0)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
        if (!split && rows_sane)
            for (int idx = threadIdx.x; idx < NR * D; idx += blockDim.x)
                if ((R0 + idx / D) / p.group < n)
                    store_out<T>(p, out_row(R0 + idx / D) * D + idx % D, __int_as_float(0x7fc00000));
        return;
    }
    if (MODE != kSuffix && seq == (int)gridDim.z - 1 && part == 0 && blockIdx.y == 0 && threadIdx.x == 0 &&
        (int64_t)qs0 + n != p.num_rows)
        atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);   // rows after the last chunk belong to no one
    if (R0 / p.group >= n)
        return;                                    // no row in this CTA
    Seen seen{0, 0, 0};
    TileOrder order{0, 0, 0};
    int t0 = start, t1 = L;
    int jb = 0, nblk = 0, ntiles = 0;
    // kMod: positions of the CTA's first and last row; the window's start for the last
    const int first_pos = L - n + R0 / p.group, last_pos = L - n + min(n - 1, (R0 + NR - 1) / p.group);
    const int low_max = kIsMod && p.mods.window > 0 ? max(0, last_pos - p.mods.window + 1) : 0;
    if constexpr (kIsMod) {
        // partitions cut the list of tiles to read; jb counts tiles of that list
        seen = seen_by(p.mods, seq, L, first_pos, last_pos);
        order = seen_tiles(seen, TB);
        t1 = seen.end;
        jb = split ? part * (p.partition_tokens / TB) : 0;
        if (split && jb >= order.count)
            return;
        ntiles = split ? min(order.count - jb, p.partition_tokens / TB) : order.count;
        nblk = ntiles * BPT;
    } else {
        if (p.partition_tokens > 0) {
            t0 += part * p.partition_tokens;
            if (t0 >= L)
                return;
            t1 = min(L, t0 + p.partition_tokens);
        }
        jb = t0 / BS;                             // partitions start on block boundaries
        nblk = (t1 > t0) ? (t1 + BS - 1) / BS - jb : 0;
        ntiles = (nblk + BPT - 1) / BPT;
    }
    auto tile_token = [&](int it) -> int {        // first token of tile it
        return kIsMod ? order(jb + it) * TB : jb * BS + it * TB;
    };
    auto block_of = [&](int i) -> int {           // block of the context: the CTA's i-th
        return kIsMod ? order(jb + i / BPT) * BPT + i % BPT : jb + i;
    };

    if (threadIdx.x == 0) {
#pragma unroll
        for (int s = 0; s < NSTAGE; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], RW);
        }
        *poison = 0;
        fence_mbar_init();
    }
    if (warp == NCW && lane == 0) {
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
    }
    __syncthreads();

    if (warp == NCW) {
        // ------------------------------------------------------------------ producer
        const int32_t* bt_row = p.block_tables + (int64_t)tseq * p.bt_stride;
        const uint64_t policy = l2_evict_first_policy();
        // the table entry of the CTA's i-th block (negative ids are one -1), or kUnseen: kMod
        // reads (and checks) only blocks that hold a seen token
        constexpr int kUnseen = -2;
        auto entry = [&](int i) -> int {
            if (i >= nblk)
                return kUnseen;
            const int b = block_of(i);
            if constexpr (kIsMod)
                if (!any_seen(seen, b * BS, min(b * BS + BS, t1)))
                    return kUnseen;
            return max(__ldg(bt_row + b), -1);
        };
        // entries 32 at a time (BPT divides 32), the next 32 in flight; kBlock: entries two
        // batches ahead, their scales one
        int next = entry(lane);
        int after = 0;
        RawScale sc{};
        if constexpr (kBlk) {
            after = entry(32 + lane);
            sc = load_scale(p, next, kvh);
        }
        bool aborted = false;
        for (int base = 0; base < nblk && !aborted; base += 32) {
            const int cur = next;
            if constexpr (kBlk) {
                scales[(base + lane) & (kScaleRing - 1)] = block_scale(sc);
                __syncwarp();
                next = after;
                sc = load_scale(p, next, kvh);
                after = entry(base + 64 + lane);
            } else {
                next = entry(base + 32 + lane);
            }
            const int cnt = min(32, nblk - base);
            for (int i = 0; i < cnt; i += BPT) {
                int pbn[BPT];
#pragma unroll
                for (int b = 0; b < BPT; ++b)
                    pbn[b] = __shfl_sync(kFullMask, cur, i + b);   // i + b <= 31
                const int it = (base + i) / BPT;
                const int stage = it % NSTAGE;
                int ok = 1;
                if (lane == 0) {
                    if (it >= NSTAGE && !mbar_wait(&empty[stage], ((it / NSTAGE) - 1) & 1)) {
                        atomicOr(p.err, PA_DEVERR_TIMEOUT);
                        ok = 0;
                    }
                    if (ok) {
                        bool all_valid = true;
                        uint32_t tx = 0;
                        bool valid[BPT];
#pragma unroll
                        for (int b = 0; b < BPT; ++b) {
                            const bool want = pbn[b] != kUnseen;
                            valid[b] = want && pbn[b] >= 0 && (int64_t)pbn[b] < p.num_blocks;
                            all_valid = all_valid && (!want || valid[b]);
                            tx += valid[b] ? 2u * BS * D * (uint32_t)sizeof(TK) : 0u;
                        }
                        stage_ok[stage] = all_valid ? 1 : 0;
                        if (!all_valid)
                            atomicOr(p.err, PA_DEVERR_BLOCK_ID);
                        if (tx == 0)
                            mbar_arrive(&full[stage]);
                        else
                            mbar_arrive_expect_tx(&full[stage], tx);
                        unsigned char* dst = smem + stage * Sm::kStageBytes;
#pragma unroll
                        for (int b = 0; b < BPT; ++b) {
                            if (!valid[b])
                                continue;
                            unsigned char* bdst = dst + b * (BS * (kFp8 ? D : 128));   // rows of block b
                            const int z = pbn[b] * p.num_kv_heads + kvh;    // < 2^31 (checked on the host)
#pragma unroll
                            for (int h = 0; h < (kFp8 ? 1 : D / 64); ++h) {
                                tma_load_3d(bdst + h * Sm::kHalfBytes, &tk, 64 * h, 0, z, &full[stage], policy);
                                tma_load_3d(bdst + Sm::kTileBytes + h * Sm::kHalfBytes, &tv, 64 * h, 0, z,
                                            &full[stage], policy);
                            }
                        }
                    }
                }
                if (!__shfl_sync(kFullMask, ok, 0)) {
                    aborted = true;
                    break;
                }
            }
        }
        return;                                   // every copy is waited for by the consumers
    }

    // ---------------------------------------------------------------------- consumers
    const int g = lane >> 2;          // fragment row: rows g and g + 8 of the warp's 16
    const int c = lane & 3;           // fragment column pair
    const int W0 = R0 + (warp % RW) * kRowsGroup;     // the warp's first row
    const bool idle = W0 / p.group >= n;              // no row of the group exists
    // per row (g, g + 8): live, and for kMod its position and the base-2 distance slope; a row
    // sees token t when t < seen.glob or position - t is in [0, reach)
    bool live[2];
    int lim[2];
    float slope[2];
    const unsigned reach = kIsMod && p.mods.window > 0 ? (unsigned)p.mods.window : 0x80000000u;
    uint32_t qa[KS][4];               // A fragments of Q
    float row_unscale[2] = {1.f, 1.f};   // bf16 rows over E4M3 caches were scaled to fit f16
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int R = W0 + g + 8 * j;
        const int tok = R / p.group;
        live[j] = tok < n;
        // (a padding row, all zeros and never stored, may see anything)
        lim[j] = kIsMod ? L - n + tok : 0;
        slope[j] = 0.f;
        if (has_slope(MODE) && live[j] && p.mods.slopes)
            slope[j] = base2_slope(p.mods.slopes[kvh * p.group + (R - tok * p.group)]);
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(reinterpret_cast<const T*>(p.q) +
                                                                 (live[j] ? out_row(R) : 0) * D);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            // k-indices 2c, 2c+1 | 2c+8, 2c+9 of step ks are head dims 16ks + 2c.. | +8.., or,
            // reading E4M3 bytes in place, 16ks + 4c, +1 | +2, +3 (K is permuted alike)
            const int d0 = kFp8 ? 16 * ks + 4 * c : 16 * ks + 2 * c;
            const int d1 = kFp8 ? d0 + 2 : d0 + 8;
            qa[ks][j] = live[j] ? __ldg(qrow + d0 / 2) : 0u;
            qa[ks][2 + j] = live[j] ? __ldg(qrow + d1 / 2) : 0u;
        }
    }
    if constexpr (kFp8 && !std::is_same_v<T, __half>) {
        // bf16 queries become f16 operands, each row scaled by a power of two (f16_row_shift)
        // that goes back into its scores
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float amax = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int k = j; k < 4; k += 2) {
                    const float2 f = Mma<T>::unpack(qa[ks][k]);
                    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
            const int sh = f16_row_shift(amax);
            const float up = __int_as_float((127 + sh) << 23);
            row_unscale[j] = __int_as_float((127 - sh) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int k = j; k < 4; k += 2) {
                    const float2 f = Mma<T>::unpack(qa[ks][k]);
                    qa[ks][k] = Mma<__half>::pack(f.x * up, f.y * up);
                }
        }
    }
    float m[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
    // O fragments of column block i: (row g, dims x, y), (row g + 8, dims x, y); x, y =
    // 8i + 2c, +1, or for E4M3 (i = 4j + k) 32j + 8c + k, + 4
    float o[NB][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[i][j] = 0.f;
    bool poisoned = false;
    // (kBlock: the K scale of each block comes with its tile)
    const float sl2 = kFp8 && !kBlk ? p.scale_log2 * p.k_scale[kvh] : p.scale_log2;
    const float row_sl2[2] = {sl2 * row_unscale[0], sl2 * row_unscale[1]};

    for (int it = warp / RW; it < ntiles; it += TW) {
        const int stage = it % NSTAGE;
        if (!mbar_wait(&full[stage], (it / NSTAGE) & 1)) {
            if (lane == 0)
                atomicOr(p.err, PA_DEVERR_TIMEOUT);
            poisoned = true;
            break;
        }
        if (!stage_ok[stage] || idle) {
            poisoned = poisoned || !idle;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[stage]);
            continue;
        }
        const uint32_t kbase = smem_addr(smem + stage * Sm::kStageBytes);
        const uint32_t vbase = kbase + Sm::kTileBytes;
        const int tb = tile_token(it);
        const int nvalid = min(TB, t1 - tb);
        // ---- S = Q . K^T: s[h] = tokens 8h .. 8h + 7 of the tile, four independent chains
        float s[4][4];
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                s[h][k] = 0.f;
        if constexpr (kFp8) {
            // token row 8h + g: the 4 codes at head dims 16ks + 4c .. +3 (chunk ks, swizzled by
            // the row; the row's low bits are g whatever h is)
            // (head_dim 64: two tokens a line, so eight rows on are four lines on, and column ^ 4)
            const uint32_t ka = kbase + e4m3_at<D>(g, 0) + 4 * c;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t w = lds_u32((ka ^ (ks << 4) ^ (D == 64 ? (h & 1) << 6 : 0)) + h * 8 * D);
                    Mma<TM>::run(s[h], qa[ks], e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
                }
        } else {
            // lane -> token row 16mb + (lane & 7) + 8 (lane >> 4) and 16-byte column 2ks + bit 3
            // of the lane; the swizzled column is that XOR the row's low bits, and 2ks is even,
            // so every address is one XOR of a lane constant
            const int r = (lane & 7) + 8 * (lane >> 4);
            const uint32_t ka = kbase + r * 128 + ((((lane >> 3) & 1) ^ (r & 7)) << 4);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int mb = 0; mb < 2; ++mb) {
                    uint32_t b[4];
                    ldsm_x4((ka ^ (((2 * ks) & 7) << 4)) + (ks >> 2) * Sm::kHalfBytes + mb * 2048, b);
                    Mma<TM>::run(s[2 * mb], qa[ks], b[0], b[1]);
                    Mma<TM>::run(s[2 * mb + 1], qa[ks], b[2], b[3]);
                }
        }
        // ---- online softmax: s[h][2j + e] = row g + 8j, token 8h + 2c + e of the tile
        float inv_v[2] = {1.f, 1.f};              // kBlock: 1 / V scale of each 16 tokens' block
        if constexpr (kBlk) {
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
                const float4 sc = scales[(it * BPT + 16 * mb / BS) & (kScaleRing - 1)];
                inv_v[mb] = sc.z;
                const float mul[2] = {row_sl2[0] * sc.x, row_sl2[1] * sc.x};
#pragma unroll
                for (int h = 2 * mb; h < 2 * mb + 2; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        s[h][k] = fmaf(s[h][k], mul[k >> 1], sc.y);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[h][k] *= row_sl2[k >> 1];
        }
        bool ragged = nvalid < TB;                // some tokens are outside, or seen by no row
        bool mask = ragged;                       // some row does not see some token
        if constexpr (kIsMod) {
            ragged = ragged || (tb < seen.lo && tb + TB > seen.glob);
            mask = !(tb + TB <= seen.glob || (tb + TB - 1 <= first_pos && tb >= low_max));
            if (has_cap(MODE) && p.mods.cap > 0.f) {
                // scores well within the cap (the usual case): the short form of tanh (only where
                // no score is of a hidden token: what such a slot holds chooses nothing)
                bool near_cap = !mask;
                if (near_cap) {
                    float far0 = 0.f;
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            far0 = fmaxf(far0, fabsf(s[h][k]));
                    near_cap = __all_sync(kFullMask, far0 * p.mods.inv_cap <= kCapNear);
                }
                if (near_cap) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            s[h][k] = cap_score_near(s[h][k], p.mods);
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            s[h][k] = cap_score(s[h][k], p.mods);
                }
            }
            if (has_slope(MODE) && p.mods.slopes) {
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        s[h][k] = fmaf(-slope[k >> 1],
                                       fabsf((float)(lim[k >> 1] - (tb + 8 * h + 2 * c + (k & 1)))), s[h][k]);
            }
        }
        if (mask) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tt = 8 * h + 2 * c + (k & 1), t = tb + tt, j = k >> 1;
                    const bool sees = kIsMod ? t < seen.glob || (unsigned)(lim[j] - t) < reach : tt < nvalid;
                    s[h][k] = sees ? s[h][k] : -INFINITY;
                }
        }
        // A row's reference maximum moves only when a tile's maximum exceeds it by more than
        // 2^8 in probability (O / l is exact for any reference), so that after the first tiles
        // O is hardly ever rescaled: with 16 rows a warp some row's true maximum rises in most
        // tiles.
        float tmax[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float a = fmaxf(fmaxf(s[0][2 * j], s[0][2 * j + 1]), fmaxf(s[1][2 * j], s[1][2 * j + 1]));
            float b = fmaxf(fmaxf(s[2][2 * j], s[2][2 * j + 1]), fmaxf(s[3][2 * j], s[3][2 * j + 1]));
            a = fmaxf(a, b);
            a = fmaxf(a, __shfl_xor_sync(kFullMask, a, 1));
            tmax[j] = fmaxf(a, __shfl_xor_sync(kFullMask, a, 2));
        }
        if (__any_sync(kFullMask, tmax[0] > m[0] + 8.f || tmax[1] > m[1] + 8.f)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (tmax[j] > m[j] + 8.f) {
                    const float alpha = ex2_approx(m[j] - tmax[j]);      // 0 on the first tile
                    m[j] = tmax[j];
                    lsum[j] *= alpha;
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        o[i][2 * j] *= alpha;
                        o[i][2 * j + 1] *= alpha;
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // a row that has seen no token yet has only -inf scores: 2^(-inf - 0) = 0
            const float ref = m[j] == -INFINITY ? 0.f : m[j];
            float sum = 0.f;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                s[h][2 * j] = ex2_approx(s[h][2 * j] - ref);
                s[h][2 * j + 1] = ex2_approx(s[h][2 * j + 1] - ref);
                if constexpr (kBlk)
                    sum = fmaf(s[h][2 * j] + s[h][2 * j + 1], inv_v[h >> 1], sum);
                else
                    sum += s[h][2 * j] + s[h][2 * j + 1];
            }
            lsum[j] += sum;
        }
        // ---- O += P . V over the two 16-token halves; V rows of tokens outside the range, or
        // that no row sees, count 0
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
            // P (hi + lo) as A fragments: rows g, g + 8 of the low 8 tokens, then of the high
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float a = s[2 * mb + (k >> 1)][2 * (k & 1)], b = s[2 * mb + (k >> 1)][2 * (k & 1) + 1];
                hi[k] = Mma<TM>::pack(a, b);
                const float2 f = Mma<TM>::unpack(hi[k]);
                lo[k] = Mma<TM>::pack(a - f.x, b - f.y);
            }
            uint32_t m01 = 0xffffffffu, m23 = 0xffffffffu;
            if (ragged) {
                auto live_tok = [&](int t) -> bool {
                    return t < nvalid && (!kIsMod || is_seen(seen, tb + t));
                };
                const int t = 16 * mb + 2 * c;
                m01 = (live_tok(t) ? 0x0000ffffu : 0u) | (live_tok(t + 1) ? 0xffff0000u : 0u);
                m23 = (live_tok(t + 8) ? 0x0000ffffu : 0u) | (live_tok(t + 9) ? 0xffff0000u : 0u);
            }
            if constexpr (kFp8) {
                // 4-byte loads of the token rows 2c, 2c+1 (+8) at dims 32j + 4g .. +3: token
                // pairs interleaved by byte_perm are the B fragments of four column blocks
                const uint32_t va = vbase + mb * 16 * D + e4m3_at<D>(2 * c, g >> 2) + 4 * (g & 3);
                // row 2c + 1: a line on and column ^ 1, or the line's other half
                const uint32_t vb = va ^ (D == 128 ? 0x90 : 0x40);
                constexpr uint32_t kEight = D == 128 ? 0 : 0x40;       // rows + 8: column ^ 4 of D / 16 lines on
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint32_t w0 = lds_u32(va ^ (j << 5));
                    const uint32_t w1 = lds_u32(vb ^ (j << 5));
                    const uint32_t w8 = lds_u32((va ^ (j << 5) ^ kEight) + 8 * D);
                    const uint32_t w9 = lds_u32((vb ^ (j << 5) ^ kEight) + 8 * D);
                    const uint32_t e01 = __byte_perm(w0, w1, 0x5140), e23 = __byte_perm(w0, w1, 0x7362);
                    const uint32_t f01 = __byte_perm(w8, w9, 0x5140), f23 = __byte_perm(w8, w9, 0x7362);
                    const uint32_t b0[4] = {e4m3x2_to_f16x2(e01), e4m3x2_to_f16x2(e01 >> 16),
                                            e4m3x2_to_f16x2(e23), e4m3x2_to_f16x2(e23 >> 16)};
                    const uint32_t b1[4] = {e4m3x2_to_f16x2(f01), e4m3x2_to_f16x2(f01 >> 16),
                                            e4m3x2_to_f16x2(f23), e4m3x2_to_f16x2(f23 >> 16)};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        Mma<TM>::run(o[4 * j + k], hi, b0[k] & m01, b1[k] & m23);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        Mma<TM>::run(o[4 * j + k], lo, b0[k] & m01, b1[k] & m23);
                }
            } else {
                const int r = (lane & 7) + 8 * ((lane >> 3) & 1);             // token row
                const uint32_t va = vbase + mb * 2048 + r * 128 + (((lane >> 4) ^ (r & 7)) << 4);
#pragma unroll
                for (int i = 0; i < NB / 2; ++i) {
                    uint32_t b[4];
                    ldsm_x4_trans((va ^ (((2 * i) & 7) << 4)) + (i >> 2) * Sm::kHalfBytes, b);
                    if (ragged) {
                        b[0] &= m01;
                        b[1] &= m23;
                        b[2] &= m01;
                        b[3] &= m23;
                    }
                    Mma<TM>::run(o[2 * i], hi, b[0], b[1]);
                    Mma<TM>::run(o[2 * i + 1], hi, b[2], b[3]);
                    Mma<TM>::run(o[2 * i], lo, b[0], b[1]);
                    Mma<TM>::run(o[2 * i + 1], lo, b[2], b[3]);
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&empty[stage]);
    }

    // ------------------------------------------------------------- merge the warps
    named_barrier(1, NCW * 32);            // every tile consumed: the ring is free
    constexpr int MR = Sm::kMergeRow;
    float* mrg_acc = reinterpret_cast<float*>(smem);                    // [NCW][16][MR]
    float* mrg_ml = mrg_acc + NCW * kRowsGroup * MR;                     // [NCW][16][2]
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float l = lsum[j];
        l += __shfl_xor_sync(kFullMask, l, 1);
        l += __shfl_xor_sync(kFullMask, l, 2);
        const int row = warp * kRowsGroup + g + 8 * j;
        if (c == 0)
            *reinterpret_cast<float2*>(mrg_ml + row * 2) = make_float2(m[j], l);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if constexpr (kFp8) {
                mrg_acc[row * MR + 32 * (i / 4) + 8 * c + i % 4] = o[i][2 * j];
                mrg_acc[row * MR + 32 * (i / 4) + 8 * c + i % 4 + 4] = o[i][2 * j + 1];
            } else {
                *reinterpret_cast<float2*>(mrg_acc + row * MR + 8 * i + 2 * c) =
                    make_float2(o[i][2 * j], o[i][2 * j + 1]);
            }
        }
    }
    if (poisoned)
        *poison = 1;
    named_barrier(1, NCW * 32);

    // TPR threads a row, each every TPR-th 4-dim piece of it
    constexpr int TPR = NCW * 32 / NR;
    const bool bad = *poison != 0;
    const int h = threadIdx.x / TPR;
    if ((R0 + h) / p.group >= n)
        return;                                        // a padding row
    // the row's warps: wt RW + (row group)
    auto part_row = [&](int wt) { return (wt * RW + h / kRowsGroup) * kRowsGroup + h % kRowsGroup; };
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < TW; ++w)
        M = fmaxf(M, mrg_ml[part_row(w) * 2]);
    float cw[TW], den = 0.f;
#pragma unroll
    for (int w = 0; w < TW; ++w) {
        const float2 ml = *reinterpret_cast<const float2*>(mrg_ml + part_row(w) * 2);
        cw[w] = M == -INFINITY ? 0.f : ex2_approx(ml.x - M);
        den = fmaf(cw[w], ml.y, den);
    }
    // no visible token gives 0; a poisoned CTA, or NaN scores, NaN
    const float vs = kFp8 && !kBlk ? p.v_scale[kvh] : 1.f;
    const float mul = bad || den != den ? __int_as_float(0x7fc00000) : den > 0.f ? vs / den : 0.f;
    const int64_t row = out_row(R0 + h);
    const int64_t prow = row * p.max_parts + (MODE == kSuffix ? p.part_base : 0) + part;
    if (split && threadIdx.x % TPR == 0)
        *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(M, den);
#pragma unroll
    for (int i = 0; i < D / 4 / TPR; ++i) {
        const int d = 4 * (threadIdx.x % TPR + i * TPR);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < TW; ++w) {
            const float4 a = *reinterpret_cast<const float4*>(mrg_acc + part_row(w) * MR + d);
            v.x = fmaf(cw[w], a.x, v.x);
            v.y = fmaf(cw[w], a.y, v.y);
            v.z = fmaf(cw[w], a.z, v.z);
            v.w = fmaf(cw[w], a.w, v.w);
        }
        v = make_float4(v.x * mul, v.y * mul, v.z * mul, v.w * mul);
        if (split || p.out_f32) {
            float* dst = split ? p.part_o + prow * D : static_cast<float*>(p.out) + row * D;
            *reinterpret_cast<float4*>(dst + d) = v;
        } else {
            *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * D + d) =
                make_uint2(Mma<T>::pack(v.x, v.y), Mma<T>::pack(v.z, v.w));
        }
    }
}

}  // namespace pa
