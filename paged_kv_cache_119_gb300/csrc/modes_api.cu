// modes_api.cu -- entry points of the attention with modified scores and of the
// shared-prefix decode (include/pa.h): argument checks, the choice of kernel and split, and
// the launches.  Host code only.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "pa.h"
#include "pa_host.h"
#include "pa_internal.h"

using namespace pa;

namespace {

enum class Family { kCore, kRows, kTc8, kChunk };

// How a pass runs: the kernel family, the (token, head) rows of a kv head one CTA serves,
// the CTAs per (sequence or group, kv head, partition), the tokens of a K/V tile, and the
// partition length (0: one pass).
struct Plan {
    Family family;
    int per;
    int chunks;
    int tile;
    int partition;
    int64_t units, slots;
};

struct Shape {
    pa_dtype q_dtype, kv_dtype;
    int num_q_heads, num_kv_heads, head_dim, block_size;
    int group() const { return num_q_heads / num_kv_heads; }
    bool fp8() const { return kv_dtype == PA_FP8_E4M3; }
};

int occupancy(const Shape& s, AttnMode mode, Family f, int per)
{
    const bool bf16 = s.q_dtype == PA_BF16;
    switch (f) {
    case Family::kCore:
        return occupancy_core_mode(mode, s.q_dtype, s.kv_dtype, s.head_dim, s.block_size, per);
    case Family::kTc8: return occupancy_tc8_mode(mode, s.q_dtype, s.block_size, per);
    case Family::kRows:
        if (s.fp8())
            return bf16 ? occupancy_rows_bf16_fp8(mode, s.head_dim, s.block_size, per)
                        : occupancy_rows_f16_fp8(mode, s.head_dim, s.block_size, per);
        return bf16 ? occupancy_rows_bf16(mode, s.head_dim, s.block_size, per)
                    : occupancy_rows_f16(mode, s.head_dim, s.block_size, per);
    case Family::kChunk:
        if (s.fp8())
            return bf16 ? occupancy_chunk_bf16_fp8(mode, s.head_dim, s.block_size)
                        : occupancy_chunk_f16_fp8(mode, s.head_dim, s.block_size);
        return bf16 ? occupancy_chunk_bf16(mode, s.head_dim, s.block_size)
                    : occupancy_chunk_f16(mode, s.head_dim, s.block_size);
    }
    return 0;
}

// Fills in the split of a plan whose pass reads at most `length` tokens for each of `count`
// sequences or groups.
void choose_split(Plan& pl, const Shape& s, AttnMode mode, int64_t count, int length,
                  int partition_size)
{
    pl.units = count * s.num_kv_heads * pl.chunks;
    pl.slots = partition_size == 0
                   ? (int64_t)device_sm_count() * occupancy(s, mode, pl.family, pl.per)
                   : 0;
    if (pl.family == Family::kTc8)
        pl.partition = choose_partition_tc8(partition_size, length, pl.units, pl.slots);
    else if (pl.family == Family::kChunk)
        pl.partition = choose_chunk_partition(partition_size, length, pl.units, pl.slots);
    else                                         // whole tiles of any family: multiples of 64
        pl.partition = choose_partition(partition_size, length, pl.units, pl.slots, 64);
}

// Rows of a kv head that a mma.sync CTA serves when there are `rows` of them: 4 or 8
// (decode_mma_kernel), 16, 32 or 64 (decode_rows_kernel; E4M3 at head_dim 64, whose tiles are
// converted warp by warp, stays at 8).
int rows_per_cta(const Shape& s, int64_t rows)
{
    if (rows <= 4)
        return 4;
    if (rows <= 8 || (s.fp8() && s.head_dim == 64))
        return 8;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// Tokens of a mma.sync kernel's tile.
int rows_tile(const Shape& s, int per)
{
    return per > 8 || (s.fp8() && s.head_dim == 128) ? 32 : s.block_size;
}

// Kernel of a pass with one row per query head of a sequence (decode, or the suffix of the
// shared-prefix decode).  Up to two heads per kv head the CUDA-core kernel streams faster
// than a 16-row matrix fragment that is mostly empty (the rule of pa_decode); E4M3 codes at
// head_dim 128 go to the tensor core as they are for up to four rows.  Other groups take
// the next of 4, 8, 16, 32 or 64 rows, padded, so that a K/V byte is read once whatever the
// group.  Capped decode of contexts up to 2048, this rule's kernel against mma.sync: f16, one head
// (64 sequences, 40 kv heads) 195 against 237 us, bf16, two heads (128, 20) 205 against 238; E4M3,
// one head 105 against 170, four heads (256, 8) 97 against 139.
Plan plan_heads(const Shape& s)
{
    Plan pl{};
    const int G = s.group();
    if (s.kv_dtype == PA_F32) {
        pl.family = Family::kCore;
        pl.per = heads_per_cta(G);
        pl.chunks = G / pl.per;
        pl.tile = s.block_size;
        return pl;
    }
    if (s.fp8() && use_tc8(s.head_dim, G)) {
        pl.family = Family::kTc8;
        pl.per = G == 3 ? 4 : G;
        pl.chunks = 1;
        pl.tile = 128;
        return pl;
    }
    if (G <= 2) {
        pl.family = Family::kCore;
        pl.per = G;
        pl.chunks = 1;
        pl.tile = s.block_size;
        return pl;
    }
    pl.family = Family::kRows;
    pl.per = rows_per_cta(s, G);
    pl.chunks = (G + pl.per - 1) / pl.per;
    pl.tile = rows_tile(s, pl.per);
    return pl;
}

// Kernel of a pass with `tokens` x group rows per kv head: at most few_rows of them (and
// E4M3 at head_dim 64, whose tiles no tensor map reaches) on a decode kernel's row mode,
// more on the tcgen05 chunk kernel.
Plan plan_rows(const Shape& s, int64_t tokens, int few_rows)
{
    Plan pl{};
    const int64_t rows = tokens * s.group();
    if (rows <= few_rows || (s.fp8() && s.head_dim != 128)) {
        pl.per = rows_per_cta(s, rows);
        pl.family = s.fp8() && use_tc8(s.head_dim, pl.per) ? Family::kTc8 : Family::kRows;
        pl.chunks = (int)std::min<int64_t>((rows + pl.per - 1) / pl.per, INT32_MAX);
        pl.tile = pl.family == Family::kTc8 ? 128 : rows_tile(s, pl.per);
        return pl;
    }
    pl.family = Family::kChunk;
    const int tt = kChunkCtaRows / s.group();    // tokens per CTA
    pl.per = tt * s.group();
    pl.chunks = (int)std::min<int64_t>((tokens + tt - 1) / tt, INT32_MAX);
    pl.tile = 64;
    return pl;
}

cudaError_t launch(const Shape& s, AttnMode mode, const Plan& pl, const DecodeParams& d,
                   const ChunkParams& c, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,
                   cudaStream_t st)
{
    const bool bf16 = s.q_dtype == PA_BF16;
    switch (pl.family) {
    case Family::kCore:
        return launch_core_mode(d, mode, s.q_dtype, s.kv_dtype, s.head_dim, s.block_size, pl.per, grid,
                                st);
    case Family::kTc8: return launch_tc8_mode(d, mode, s.q_dtype, s.block_size, pl.per, tk, tv, grid, st);
    case Family::kRows:
        if (s.fp8())
            return (bf16 ? launch_rows_bf16_fp8 : launch_rows_f16_fp8)(d, mode, s.head_dim, s.block_size,
                                                                       pl.per, tk, tv, grid, st);
        return (bf16 ? launch_rows_bf16 : launch_rows_f16)(d, mode, s.head_dim, s.block_size, pl.per, tk,
                                                           tv, grid, st);
    case Family::kChunk:
        if (s.fp8())
            return (bf16 ? launch_chunk_bf16_fp8 : launch_chunk_f16_fp8)(c, mode, s.head_dim,
                                                                         s.block_size, tk, tv, grid, st);
        return (bf16 ? launch_chunk_bf16 : launch_chunk_f16)(c, mode, s.head_dim, s.block_size, tk, tv,
                                                             grid, st);
    }
    return cudaErrorInvalidValue;
}

// Tensor maps of both caches where a kernel of this shape wants them.
cudaError_t maps(const Shape& s, const void* k_cache, const void* v_cache, int64_t num_blocks,
                 CUtensorMap* tk, CUtensorMap* tv)
{
    if (s.kv_dtype == PA_F32 || (s.fp8() && s.head_dim != 128))
        return cudaSuccess;                      // 1-D bulk copies
    cudaError_t e = kv_tensor_map(tk, k_cache, num_blocks, s.num_kv_heads, s.block_size, s.head_dim,
                                  s.kv_dtype);
    if (e == cudaSuccess)
        e = kv_tensor_map(tv, v_cache, num_blocks, s.num_kv_heads, s.block_size, s.head_dim, s.kv_dtype);
    return e;
}

// Checks common to both calls; a positive value means "go on".
int check_shape(const Shape& s, pa_dtype out_dtype, const float* k_scale, const float* v_scale,
                int64_t num_blocks, int64_t block_table_stride, int64_t num_seqs, float scale,
                int partition_size)
{
    if (!(s.q_dtype == PA_F32 || s.q_dtype == PA_F16 || s.q_dtype == PA_BF16) ||
        !(out_dtype == PA_F32 || out_dtype == s.q_dtype))
        return PA_ERR_INVALID;
    if (num_seqs < 0 || num_seqs > 65535 || s.num_q_heads <= 0 || s.num_kv_heads <= 0 ||
        s.num_q_heads % s.num_kv_heads != 0 || s.num_q_heads > 65535)
        return PA_ERR_INVALID;
    if (!(s.head_dim == 64 || s.head_dim == 128) || !(s.block_size == 16 || s.block_size == 32))
        return PA_ERR_UNSUPPORTED;
    if (s.fp8() && s.q_dtype == PA_F32)
        return PA_ERR_UNSUPPORTED;
    if (num_blocks <= 0 || num_blocks > INT32_MAX || block_table_stride <= 0 || !std::isfinite(scale) ||
        (partition_size > 0 && partition_size % 128 != 0))
        return PA_ERR_INVALID;
    if (num_blocks * s.num_kv_heads >= (int64_t(1) << 31))   // a tile's index is 32-bit
        return PA_ERR_INVALID;
    if (s.fp8() && (!k_scale || !v_scale))
        return PA_ERR_INVALID;
    return 1;
}

constexpr int kMaxContext = 1 << 30;             // positions and their sums stay in int32

struct Buffers {
    void* out;
    size_t out_bytes;
    Span spans[9];
    int n = 0;
    void add(const void* p, size_t bytes)
    {
        if (p)
            spans[n++] = {p, bytes};
    }
    // out and the workspace touch none of the inputs, and not each other
    bool out_clear() const
    {
        for (int i = 0; i < n; ++i)
            if (overlaps(out, out_bytes, spans[i].p, spans[i].n))
                return false;
        return true;
    }
    bool clear(const void* ws, size_t bytes) const
    {
        for (int i = 0; i < n; ++i)
            if (overlaps(ws, bytes, spans[i].p, spans[i].n))
                return false;
        return !overlaps(ws, bytes, out, out_bytes);
    }
};

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Most tokens a CTA of a kMod pass can have to read, in whole tiles.
int64_t seen_bound(int max_context_len, int window, int max_global, int query_len, int tile)
{
    const int64_t all = ((int64_t)max_context_len + tile - 1) / tile * tile;
    if (window == 0)
        return all;
    // a run of n tokens touches at most (n + tile - 2) / tile + 1 tiles
    const int64_t run = (int64_t)window + query_len - 1;
    const int64_t tiles = (std::min(max_global, max_context_len) + (int64_t)tile - 1) / tile +
                          (run + tile - 2) / tile + 1;
    return std::min(all, tiles * tile);
}

// Shared body of the four modified-score calls; query_start null: decode (one row per
// sequence, num_query_tokens = num_seqs).
int mod_impl(bool decode, void* out, pa_dtype out_dtype, const void* q, const Shape& s,
             const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
             int64_t num_blocks, const int32_t* block_tables, int64_t block_table_stride,
             const int32_t* context_lens, const int32_t* query_start, int64_t num_query_tokens,
             int32_t max_query_len, int32_t max_context_len, int32_t num_seqs, float scale,
             float softcap, const float* alibi_slopes, int32_t window, const int32_t* global_lens,
             int32_t max_global_len, int32_t partition_size, void* workspace, size_t workspace_bytes,
             void* stream)
{
    const int ok = check_shape(s, out_dtype, k_scale, v_scale, num_blocks, block_table_stride, num_seqs,
                               scale, partition_size);
    if (ok <= 0)
        return ok;
    if (!decode && (s.q_dtype == PA_F32 || s.group() > 128))
        return s.q_dtype == PA_F32 ? PA_ERR_UNSUPPORTED : PA_ERR_INVALID;
    if (max_context_len < 0 || max_context_len > kMaxContext ||
        (int64_t)max_context_len > block_table_stride * s.block_size || max_query_len < 0 ||
        max_query_len > max_context_len || num_query_tokens < 0 || num_query_tokens > INT32_MAX)
        return PA_ERR_INVALID;
    // the cap's reciprocal and its base-2 form stay normal numbers
    if (!(softcap == 0.f || (softcap >= 1e-30f && softcap <= 1e30f)) || window < 0 || max_global_len < 0)
        return PA_ERR_INVALID;
    if (num_seqs == 0 || num_query_tokens == 0 || (!decode && max_query_len == 0))
        return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || (!decode && !query_start))
        return PA_ERR_INVALID;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned4(alibi_slopes) || !aligned4(global_lens) || !aligned4(block_tables) ||
        !aligned4(context_lens) || !aligned4(query_start) || !aligned4(k_scale) || !aligned4(v_scale))
        return PA_ERR_INVALID;
    if (!global_lens)
        max_global_len = 0;
    const int qlen = decode ? 1 : max_query_len;
    // (32 rows of a chunk on a decode kernel's row mode against the chunk kernel, 32 sequences,
    // capped: 35.1 against 49.3 us over a window of 1024, 198 against 278 over 8192 tokens; 64 rows
    // 60.2 against 51.4 and 377 against 280)
    Plan pl = decode ? plan_heads(s) : plan_rows(s, qlen, kChunkRowsMax);
    AttnMode mode = kMod;
    const bool cap = softcap > 0.f, slope = alibi_slopes != nullptr;
    if (pl.family == Family::kChunk)
        mode = cap ? (slope ? kModBoth : kModCap) : (slope ? kModSlope : kMod);
    else if (pl.family == Family::kRows)
        mode = cap || slope ? kModBoth : kMod;
    const int length =
        (int)std::min<int64_t>(seen_bound(max_context_len, window, max_global_len, qlen, pl.tile), INT32_MAX);
    choose_split(pl, s, mode, num_seqs, length, partition_size);
    if ((int64_t)s.num_kv_heads * pl.chunks > 65535 || pl.units > INT32_MAX / 64)
        return PA_ERR_INVALID;

    Buffers b;
    const size_t row_elems = (size_t)num_query_tokens * s.num_q_heads * s.head_dim;
    const size_t pool = (size_t)num_blocks * s.num_kv_heads * s.block_size * s.head_dim * elem_size(s.kv_dtype);
    b.out = out;
    b.out_bytes = row_elems * elem_size(out_dtype);
    b.add(q, row_elems * elem_size(s.q_dtype));
    b.add(k_cache, pool);
    b.add(v_cache, pool);
    b.add(block_tables, (size_t)num_seqs * block_table_stride * 4);
    b.add(context_lens, (size_t)num_seqs * 4);
    b.add(query_start, (size_t)(num_seqs + 1) * 4);
    b.add(alibi_slopes, (size_t)s.num_q_heads * 4);
    b.add(global_lens, (size_t)num_seqs * 4);
    if (!b.out_clear())
        return PA_ERR_INVALID;

    DecodeParams d{};
    d.out = out;
    d.q = q;
    d.k_cache = k_cache;
    d.v_cache = v_cache;
    d.block_tables = block_tables;
    d.context_lens = context_lens;
    d.query_start = query_start;
    d.num_rows = num_query_tokens;
    d.max_query_len = qlen;
    d.k_scale = s.fp8() ? k_scale : nullptr;
    d.v_scale = s.fp8() ? v_scale : nullptr;
    d.num_blocks = num_blocks;
    d.bt_stride = block_table_stride;
    d.num_seqs = num_seqs;
    d.num_q_heads = s.num_q_heads;
    d.num_kv_heads = s.num_kv_heads;
    d.group = s.group();
    d.chunks = pl.chunks;
    d.rows_per_cta = pl.per;
    d.max_context_len = max_context_len;
    d.max_parts = 1;
    d.out_f32 = out_dtype == PA_F32 ? 1 : 0;
    d.scale_log2 = (float)((double)scale * 1.4426950408889634);
    d.mods.slopes = alibi_slopes;
    d.mods.global_lens = global_lens;
    d.mods.window = window;
    d.mods.max_global = max_global_len;
    if (softcap > 0.f) {
        d.mods.cap = (float)((double)softcap * 1.4426950408889634);
        d.mods.inv_cap = 1.f / d.mods.cap;
    }
    // A one-pass grid of the chunk kernel (one CTA per SM) whose last wave is at most half full
    // leaves the rest of the SMs idle for as long as a CTA runs: its units are then cut into as
    // many parts as fill that wave.  4 x 512 tokens of 8192, 64/8 heads, capped: 512 units on 152
    // SMs, the last 56 in two parts, 673 -> 574 us.  Without a workspace the call runs unsplit.
    int64_t whole_units = 0;
    if (pl.family == Family::kChunk && pl.partition == 0 && partition_size == 0 && pl.slots > 0) {
        const int64_t rest = pl.units % pl.slots;
        const int64_t cut = rest > 0 && pl.units > pl.slots ? std::min(pl.slots / rest, (int64_t)length / 512) : 0;
        const int64_t P = cut > 1 ? ((length + cut - 1) / cut + 63) / 64 * 64 : 0;
        const int64_t parts = P > 0 ? (length + P - 1) / P : 0;
        const size_t need = parts > 1 ? workspace_layout(num_query_tokens * s.num_q_heads, (int)parts,
                                                         s.head_dim, nullptr)
                                      : 0;
        if (need > 0 && workspace && workspace_bytes >= need && aligned16(workspace) &&
            b.clear(workspace, need)) {
            whole_units = pl.units - rest;
            pl.partition = (int)P;
        }
    }
    d.partition_tokens = pl.partition;
    d.whole_units = (int)whole_units;
    if (pl.partition > 0) {
        d.max_parts = (length + pl.partition - 1) / pl.partition;
        size_t ml_off = 0;
        const size_t need =
            workspace_layout(num_query_tokens * s.num_q_heads, d.max_parts, s.head_dim, &ml_off);
        if (!workspace || workspace_bytes < need || !aligned16(workspace))
            return PA_ERR_WORKSPACE;
        if (!b.clear(workspace, need))
            return PA_ERR_INVALID;
        d.part_o = static_cast<float*>(workspace);
        d.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml_off);
    }
    const int64_t ctas = whole_units + (pl.units - whole_units) * d.max_parts;
    if (ctas > INT32_MAX)                        // (one-dimensional grid of the chunk kernel)
        return PA_ERR_INVALID;
    d.err = device_error_word();
    if (!d.err)
        return PA_ERR_CUDA;
    CUtensorMap tk{}, tv{};
    cudaError_t e = pl.family == Family::kCore
                        ? cudaSuccess
                        : maps(s, k_cache, v_cache, num_blocks, &tk, &tv);
    if (e != cudaSuccess)
        return e == cudaErrorInvalidValue ? PA_ERR_INVALID : PA_ERR_CUDA;

    ChunkParams c{};
    c.out = out;
    c.q = q;
    c.block_tables = block_tables;
    c.context_lens = context_lens;
    c.query_start = query_start;
    c.part_o = d.part_o;
    c.part_ml = d.part_ml;
    c.k_scale = d.k_scale;
    c.v_scale = d.v_scale;
    c.err = d.err;
    c.num_blocks = num_blocks;
    c.bt_stride = block_table_stride;
    c.num_rows = num_query_tokens;
    c.num_seqs = num_seqs;
    c.num_q_heads = s.num_q_heads;
    c.num_kv_heads = s.num_kv_heads;
    c.group = s.group();
    c.rows_tokens = pl.family == Family::kChunk ? pl.per / s.group() : 0;
    c.m_tiles = pl.chunks;
    c.max_query_len = qlen;
    c.max_context_len = max_context_len;
    c.partition_tokens = pl.partition;
    c.max_parts = d.max_parts;
    c.out_f32 = d.out_f32;
    c.scale_log2 = d.scale_log2;
    c.mods = d.mods;
    c.whole_units = d.whole_units;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // a one-pass CUDA-core grid of several waves starts the longest sequences first, as
    // pa_decode does (with a window every sequence is about as long)
    const size_t order_bytes = seq_order_bytes(num_seqs);
    if (decode && pl.family == Family::kCore && pl.partition == 0 && partition_size == 0 && window == 0 &&
        pl.slots > 0 && pl.units > pl.slots && workspace && aligned16(workspace) &&
        workspace_bytes >= order_bytes && b.clear(workspace, order_bytes)) {
        int2* order = static_cast<int2*>(workspace);
        if (launch_seq_order(context_lens, num_seqs, max_context_len, order, st) != cudaSuccess)
            return PA_ERR_CUDA;
        d.seq_order = order;
    }
    const dim3 grid = pl.family == Family::kChunk
                          ? dim3((unsigned)ctas)
                          : dim3(d.max_parts, s.num_kv_heads * pl.chunks, num_seqs);
    e = launch(s, mode, pl, d, c, tk, tv, grid, st);
    if (e == cudaSuccess && pl.partition > 0)
        e = launch_mod_merge(d, s.q_dtype, s.head_dim, pl.tile, st);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// (sequence, head) rows per kv head up to which the pass over a shared prefix runs on a decode
// kernel's row mode; the whole call, row mode against chunk kernel, bf16 / E4M3 caches, 32/8
// heads, up to 128 own tokens a sequence:
//   24 rows x 16 groups over 1024 tokens   27.6 against 31.6, 30.8 against 34.6 us
//   32 rows x 16 groups over 4096          60.5 against 72.2, 67.3 against 76.7
//   48 rows x 16 groups over 1024          41.9 against 39.7, 51.1 against 47.8
//   64 rows x 8 groups over 4096           57.0 against 50.2, 67.2 against 55.5
constexpr int kPrefixRowsMax = 32;

// The two passes of a shared-prefix decode.
struct PrefixPlan {
    Plan prefix, suffix;
    int prefix_parts, suffix_parts;
};

PrefixPlan prefix_plan(const Shape& s, int num_seqs, int num_groups, int max_group_size,
                       int max_prefix_len, int max_suffix_len, int partition_size)
{
    PrefixPlan p{};
    p.prefix = plan_rows(s, max_group_size, kPrefixRowsMax);
    choose_split(p.prefix, s, kPrefix, num_groups, max_prefix_len, partition_size);
    p.suffix = plan_heads(s);
    choose_split(p.suffix, s, kSuffix, num_seqs, max_suffix_len, partition_size);
    auto parts = [](int len, int part) { return part > 0 ? (len + part - 1) / part : (len > 0 ? 1 : 0); };
    p.prefix_parts = parts(max_prefix_len, p.prefix.partition);
    p.suffix_parts = parts(max_suffix_len, p.suffix.partition);
    return p;
}

int prefix_impl(void* out, pa_dtype out_dtype, const void* q, const Shape& s, const void* k_cache,
                const void* v_cache, const float* k_scale, const float* v_scale, int64_t num_blocks,
                const int32_t* block_tables, int64_t block_table_stride, const int32_t* context_lens,
                const int32_t* prefix_lens, const int32_t* group_start, int32_t num_groups,
                int32_t max_group_size, int32_t max_prefix_len, int32_t max_suffix_len, int32_t num_seqs,
                float scale, int32_t partition_size, void* workspace, size_t workspace_bytes, void* stream)
{
    if (s.q_dtype == PA_F32)
        return PA_ERR_UNSUPPORTED;
    const int ok = check_shape(s, out_dtype, k_scale, v_scale, num_blocks, block_table_stride, num_seqs,
                               scale, partition_size);
    if (ok <= 0)
        return ok;
    // (the suffix grid has one z-slice more than sequences)
    if (s.group() > 128 || num_seqs > 65534 || max_prefix_len < 0 || max_suffix_len < 0 ||
        (int64_t)max_prefix_len + max_suffix_len > kMaxContext)
        return PA_ERR_INVALID;
    if (max_prefix_len % s.block_size != 0 || max_prefix_len > block_table_stride * s.block_size)
        return PA_ERR_INVALID;
    if (num_groups < 0 || num_groups > num_seqs || max_group_size < 0 || max_group_size > num_seqs ||
        (num_seqs > 0 && (num_groups == 0 || max_group_size == 0)))
        return PA_ERR_INVALID;
    if (num_seqs == 0)
        return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !prefix_lens || !group_start)
        return PA_ERR_INVALID;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(prefix_lens) ||
        !aligned4(group_start) || !aligned4(k_scale) || !aligned4(v_scale))
        return PA_ERR_INVALID;
    const PrefixPlan pl = prefix_plan(s, num_seqs, num_groups, max_group_size, max_prefix_len,
                                      max_suffix_len, partition_size);
    if ((int64_t)s.num_kv_heads * std::max(pl.prefix.chunks, pl.suffix.chunks) > 65535)
        return PA_ERR_INVALID;

    Buffers b;
    const size_t row_elems = (size_t)num_seqs * s.num_q_heads * s.head_dim;
    const size_t pool = (size_t)num_blocks * s.num_kv_heads * s.block_size * s.head_dim * elem_size(s.kv_dtype);
    b.out = out;
    b.out_bytes = row_elems * elem_size(out_dtype);
    b.add(q, row_elems * elem_size(s.q_dtype));
    b.add(k_cache, pool);
    b.add(v_cache, pool);
    b.add(block_tables, (size_t)num_seqs * block_table_stride * 4);
    b.add(context_lens, (size_t)num_seqs * 4);
    b.add(prefix_lens, (size_t)num_seqs * 4);
    b.add(group_start, (size_t)(num_groups + 1) * 4);
    if (!b.out_clear())
        return PA_ERR_INVALID;
    const int max_parts = std::max(1, pl.prefix_parts + pl.suffix_parts);
    size_t ml_off = 0;
    const size_t need = workspace_layout((int64_t)num_seqs * s.num_q_heads, max_parts, s.head_dim, &ml_off);
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
        return PA_ERR_WORKSPACE;
    if (!b.clear(workspace, need))
        return PA_ERR_INVALID;

    DecodeParams d{};
    d.out = out;
    d.q = q;
    d.k_cache = k_cache;
    d.v_cache = v_cache;
    d.block_tables = block_tables;
    d.context_lens = context_lens;
    d.prefix_lens = prefix_lens;
    d.part_o = static_cast<float*>(workspace);
    d.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml_off);
    d.k_scale = s.fp8() ? k_scale : nullptr;
    d.v_scale = s.fp8() ? v_scale : nullptr;
    d.num_blocks = num_blocks;
    d.bt_stride = block_table_stride;
    d.num_seqs = num_seqs;
    d.num_rows = num_seqs;
    d.num_q_heads = s.num_q_heads;
    d.num_kv_heads = s.num_kv_heads;
    d.group = s.group();
    d.max_context_len = (int)std::min<int64_t>((int64_t)max_prefix_len + max_suffix_len,
                                               block_table_stride * s.block_size);
    d.max_prefix_len = max_prefix_len;
    d.max_suffix_len = max_suffix_len;
    d.tile_align = s.block_size;
    d.max_parts = max_parts;
    d.part_base = pl.prefix_parts;
    d.out_f32 = out_dtype == PA_F32 ? 1 : 0;
    d.scale_log2 = (float)((double)scale * 1.4426950408889634);
    d.err = device_error_word();
    if (!d.err)
        return PA_ERR_CUDA;
    CUtensorMap tk{}, tv{};
    cudaError_t e = maps(s, k_cache, v_cache, num_blocks, &tk, &tv);
    if (e != cudaSuccess)
        return e == cudaErrorInvalidValue ? PA_ERR_INVALID : PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);

    if (pl.prefix_parts > 0) {
        DecodeParams dp = d;
        dp.query_start = group_start;
        dp.max_query_len = max_group_size;
        dp.chunks = pl.prefix.chunks;
        dp.partition_tokens = pl.prefix.partition;
        ChunkParams c{};
        c.q = q;
        c.block_tables = block_tables;
        c.prefix_lens = prefix_lens;
        c.query_start = group_start;
        c.part_o = d.part_o;
        c.part_ml = d.part_ml;
        c.k_scale = d.k_scale;
        c.v_scale = d.v_scale;
        c.err = d.err;
        c.num_blocks = num_blocks;
        c.bt_stride = block_table_stride;
        c.num_rows = num_seqs;
        c.num_seqs = num_groups;
        c.num_q_heads = s.num_q_heads;
        c.num_kv_heads = s.num_kv_heads;
        c.group = s.group();
        c.rows_tokens = pl.prefix.family == Family::kChunk ? pl.prefix.per / s.group() : 0;
        c.m_tiles = pl.prefix.chunks;
        c.max_query_len = max_group_size;
        c.max_context_len = max_prefix_len;
        c.partition_tokens = pl.prefix.partition;
        c.max_parts = max_parts;
        c.scale_log2 = d.scale_log2;
        e = launch(s, kPrefix, pl.prefix, dp, c, tk, tv,
                   dim3(pl.prefix_parts, s.num_kv_heads * pl.prefix.chunks, num_groups), st);
        if (e != cudaSuccess)
            return PA_ERR_CUDA;
    }
    d.chunks = pl.suffix.chunks;
    d.partition_tokens = pl.suffix.partition;
    d.overlap = pl.prefix_parts > 0 ? 1 : 0;
    if (pl.suffix_parts > 0) {
        e = launch(s, kSuffix, pl.suffix, d, ChunkParams{}, tk, tv,
                   dim3(pl.suffix_parts, s.num_kv_heads * pl.suffix.chunks, num_seqs + d.overlap), st);
        if (e != cudaSuccess)
            return PA_ERR_CUDA;
    }
    e = launch_prefix_merge(d, s.q_dtype, s.head_dim, group_start, num_groups, max_group_size,
                            pl.prefix.partition, pl.prefix_parts + pl.suffix_parts > 0, st);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

int pa_decode_mod(void* out, pa_dtype out_dtype, const void* q, const void* k_cache,
                  const void* v_cache, pa_dtype kv_dtype, int64_t num_blocks,
                  const int32_t* block_tables, int64_t block_table_stride,
                  const int32_t* context_lens, int32_t max_context_len, int32_t num_seqs,
                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                  float scale, float softcap, const float* alibi_slopes, int32_t window,
                  const int32_t* global_lens, int32_t max_global_len, int32_t partition_size,
                  void* workspace, size_t workspace_bytes, void* stream)
{
    if (!valid_dtype(kv_dtype))
        return PA_ERR_INVALID;
    return mod_impl(true, out, out_dtype, q,
                    Shape{kv_dtype, kv_dtype, num_q_heads, num_kv_heads, head_dim, block_size}, k_cache,
                    v_cache, nullptr, nullptr, num_blocks, block_tables, block_table_stride, context_lens,
                    nullptr, num_seqs, 0, max_context_len, num_seqs, scale, softcap, alibi_slopes,
                    window, global_lens, max_global_len, partition_size, workspace, workspace_bytes,
                    stream);
}

int pa_decode_mod_fp8(void* out, pa_dtype out_dtype, const void* q, pa_dtype q_dtype,
                      const void* k_cache, const void* v_cache, const float* k_scale,
                      const float* v_scale, int64_t num_blocks, const int32_t* block_tables,
                      int64_t block_table_stride, const int32_t* context_lens,
                      int32_t max_context_len, int32_t num_seqs, int32_t num_q_heads,
                      int32_t num_kv_heads, int32_t head_dim, int32_t block_size, float scale,
                      float softcap, const float* alibi_slopes, int32_t window,
                      const int32_t* global_lens, int32_t max_global_len, int32_t partition_size,
                      void* workspace, size_t workspace_bytes, void* stream)
{
    return mod_impl(true, out, out_dtype, q,
                    Shape{q_dtype, PA_FP8_E4M3, num_q_heads, num_kv_heads, head_dim, block_size}, k_cache,
                    v_cache, k_scale, v_scale, num_blocks, block_tables, block_table_stride, context_lens,
                    nullptr, num_seqs, 0, max_context_len, num_seqs, scale, softcap, alibi_slopes,
                    window, global_lens, max_global_len, partition_size, workspace, workspace_bytes,
                    stream);
}

int pa_chunk_attention_mod(void* out, pa_dtype out_dtype, const void* q, const void* k_cache,
                           const void* v_cache, pa_dtype kv_dtype, int64_t num_blocks,
                           const int32_t* block_tables, int64_t block_table_stride,
                           const int32_t* context_lens, const int32_t* query_start,
                           int64_t num_query_tokens, int32_t max_query_len, int32_t max_context_len,
                           int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                           int32_t head_dim, int32_t block_size, float scale, float softcap,
                           const float* alibi_slopes, int32_t window, const int32_t* global_lens,
                           int32_t max_global_len, int32_t partition_size, void* workspace,
                           size_t workspace_bytes, void* stream)
{
    if (kv_dtype == PA_FP8_E4M3)
        return PA_ERR_UNSUPPORTED;               // E4M3 caches: pa_chunk_attention_mod_fp8
    return mod_impl(false, out, out_dtype, q,
                    Shape{kv_dtype, kv_dtype, num_q_heads, num_kv_heads, head_dim, block_size}, k_cache,
                    v_cache, nullptr, nullptr, num_blocks, block_tables, block_table_stride, context_lens,
                    query_start, num_query_tokens, max_query_len, max_context_len, num_seqs, scale,
                    softcap, alibi_slopes, window, global_lens, max_global_len, partition_size, workspace,
                    workspace_bytes, stream);
}

int pa_chunk_attention_mod_fp8(void* out, pa_dtype out_dtype, const void* q, pa_dtype q_dtype,
                               const void* k_cache, const void* v_cache, const float* k_scale,
                               const float* v_scale, int64_t num_blocks, const int32_t* block_tables,
                               int64_t block_table_stride, const int32_t* context_lens,
                               const int32_t* query_start, int64_t num_query_tokens,
                               int32_t max_query_len, int32_t max_context_len, int32_t num_seqs,
                               int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, float scale, float softcap,
                               const float* alibi_slopes, int32_t window, const int32_t* global_lens,
                               int32_t max_global_len, int32_t partition_size, void* workspace,
                               size_t workspace_bytes, void* stream)
{
    return mod_impl(false, out, out_dtype, q,
                    Shape{q_dtype, PA_FP8_E4M3, num_q_heads, num_kv_heads, head_dim, block_size}, k_cache,
                    v_cache, k_scale, v_scale, num_blocks, block_tables, block_table_stride, context_lens,
                    query_start, num_query_tokens, max_query_len, max_context_len, num_seqs, scale,
                    softcap, alibi_slopes, window, global_lens, max_global_len, partition_size, workspace,
                    workspace_bytes, stream);
}

size_t pa_decode_prefix_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t head_dim,
                                        int32_t max_prefix_len, int32_t max_suffix_len,
                                        int32_t partition_size)
{
    if (num_seqs < 0 || num_q_heads <= 0 || head_dim <= 0 || max_prefix_len < 0 || max_suffix_len < 0)
        return 0;
    const int P = partition_size > 0 ? partition_size : kAutoPartitionTokens;
    auto parts = [&](int len) {
        return partition_size < 0 ? (len > 0 ? 1 : 0) : (int)(((int64_t)len + P - 1) / P);
    };
    return workspace_layout((int64_t)num_seqs * num_q_heads,
                            std::max(1, parts(max_prefix_len) + parts(max_suffix_len)), head_dim, nullptr);
}

int pa_decode_prefix(void* out, pa_dtype out_dtype, const void* q, const void* k_cache,
                     const void* v_cache, pa_dtype kv_dtype, int64_t num_blocks,
                     const int32_t* block_tables, int64_t block_table_stride,
                     const int32_t* context_lens, const int32_t* prefix_lens,
                     const int32_t* group_start, int32_t num_groups, int32_t max_group_size,
                     int32_t max_prefix_len, int32_t max_suffix_len, int32_t num_seqs,
                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     float scale, int32_t partition_size, void* workspace, size_t workspace_bytes,
                     void* stream)
{
    if (!valid_dtype(kv_dtype))
        return kv_dtype == PA_FP8_E4M3 ? PA_ERR_UNSUPPORTED : PA_ERR_INVALID;
    return prefix_impl(out, out_dtype, q,
                       Shape{kv_dtype, kv_dtype, num_q_heads, num_kv_heads, head_dim, block_size}, k_cache,
                       v_cache, nullptr, nullptr, num_blocks, block_tables, block_table_stride,
                       context_lens, prefix_lens, group_start, num_groups, max_group_size, max_prefix_len,
                       max_suffix_len, num_seqs, scale, partition_size, workspace, workspace_bytes,
                       stream);
}

int pa_decode_prefix_fp8(void* out, pa_dtype out_dtype, const void* q, pa_dtype q_dtype,
                         const void* k_cache, const void* v_cache, const float* k_scale,
                         const float* v_scale, int64_t num_blocks, const int32_t* block_tables,
                         int64_t block_table_stride, const int32_t* context_lens,
                         const int32_t* prefix_lens, const int32_t* group_start, int32_t num_groups,
                         int32_t max_group_size, int32_t max_prefix_len, int32_t max_suffix_len,
                         int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, float scale, int32_t partition_size,
                         void* workspace, size_t workspace_bytes, void* stream)
{
    return prefix_impl(out, out_dtype, q,
                       Shape{q_dtype, PA_FP8_E4M3, num_q_heads, num_kv_heads, head_dim, block_size},
                       k_cache, v_cache, k_scale, v_scale, num_blocks, block_tables, block_table_stride,
                       context_lens, prefix_lens, group_start, num_groups, max_group_size, max_prefix_len,
                       max_suffix_len, num_seqs, scale, partition_size, workspace, workspace_bytes,
                       stream);
}

}  // extern "C"
