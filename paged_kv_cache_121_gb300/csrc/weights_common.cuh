// Arguments of the kernels around attention weights: the weights that decode
// steps and prompts gave the cached tokens (decode_weights.cu,
// prefill_weights_simt.cu, prefill_weights_tc.cu), and the eviction that goes by
// them (evict.cu).
#pragma once

#include "device_common.cuh"

namespace pa {

// One decode step that leaves the weight it gave each cached token.
struct DecodeWeightsParams {
    const void *query;            // [num_seqs, num_heads, head_dim]
    const void *k_cache, *v_cache;
    const int32_t *block_tables, *context_lens;
    void *out;                    // [num_seqs, num_heads, head_dim]
    float *weights;               // [num_seqs, num_kv_heads, weights_stride]
    float *scores;                // [num_seqs, num_heads, score_stride]: scale * q.k * log2(e)
    int64_t weights_stride;
    int64_t score_stride;         // a multiple of 16
    int num_seqs, num_heads, num_kv_heads, group;
    int block_size, max_blocks, num_blocks;
    int max_ctx;
    int heads_per_cta, sets;      // KV heads of a CTA, warps that share each
    int nsplit, part_tokens;      // CTAs (one cluster) and tokens each of a context
    int out_type;
    float scale_log2, decay;
};

// Division of 0 <= n < 2^31 by a number known ahead, d <= 2^16: n * m >> (31 + s) with s = ceil(log2 d) and
// m = floor(2^(31 + s) / d) + 1 (Granlund and Montgomery, "Division by invariant integers using multiplication").
struct FixedDivisor {
    uint32_t m;
    int s;
    void set(int d) {
        s = 0;
        while ((1 << s) < d) ++s;
        m = static_cast<uint32_t>((uint64_t(1) << (31 + s)) / d + 1);
    }
    __device__ __forceinline__ int of(int n) const {
        return s == 0 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), m) >> (s - 1));
    }
};

// The weights that several query tokens a sequence gave each cached token, without their outputs.
// A sequence's rows are the (query token, query head) pairs of one KV head that count, token by token.
struct PrefillWeightsParams {
    const void *query;            // [num_tokens, num_heads, head_dim]
    const void *k_cache;
    const int32_t *block_tables, *context_lens, *query_start;
    float *weights;               // [num_seqs, num_kv_heads, weights_stride]
    float2 *rows;                 // [stat_rows][num_heads]: a row's score that weighs most and 1 / sum (see row_stats)
    float *offsets;               //   the same in one number, where that will do (prefill_weights_tc; see folded_stats)
    float2 *stats;                // nsplit > 1: [nsplit][stat_rows][num_heads] maximum and sum of each piece
    int *counter;                 // prefill_weights_tc: units of the second pass drawn beyond one a CTA
    int *order;                   //   its units (one KV head's), longest first, or null (as they are numbered)
    float *parts;                 //   row_pieces > 1: [row_pieces][num_seqs][num_kv_heads][max_ctx] sums over pieces of the rows
    int64_t weights_stride, stat_rows;
    int *status;
    int num_seqs, num_tokens, num_heads, num_kv_heads, group;
    FixedDivisor group_div;       // by group
    int block_size, max_blocks, num_blocks;
    int max_count, max_ctx;       // host bounds: query tokens that count, context tokens
    int window;                   // the last so many query tokens count (0: all)
    int compact;                  // stat rows are sequence * max_count + i, else the query token's index
    int nsplit;                   // pieces of a context that a row's statistics are made in
    int pieces, pair;             // prefill_weights_tc: ranges of keys a unit of rows is cut into; 1: a unit is two
                                  //   row tiles, else one whose two halves of each range make a piece each
    int row_pieces;               // ranges of rows that a unit of keys is cut into
    float scale_log2, decay;      // (scale_log2 is not zero: masked scores are infinities ahead of it)
};

// One sequence's extent, clamped so that no index leaves its array whatever the device-side lengths hold.
struct WeightSeq {
    int q0, count;      // first query token that counts, how many
    int ctx;            // context tokens
    int past;           // context tokens ahead of the first one that counts (negative: leading rows see nothing)
    int fresh;          // tokens from here on are the call's own: their weights start here
    int64_t stat0;      // the first one's row of statistics
    __device__ int sees(int i) const {   // context tokens that counted query token i sees
        const int64_t n = static_cast<int64_t>(past) + i + 1;
        return n < 0 ? 0 : n < ctx ? static_cast<int>(n) : ctx;
    }
};

__device__ __forceinline__ WeightSeq weight_seq(const PrefillWeightsParams &p, int b) {
    WeightSeq s;
    const int start = p.query_start[b];
    const int64_t given = static_cast<int64_t>(p.query_start[b + 1]) - start;
    int64_t n = given;
    if (start < 0 || start > p.num_tokens) n = 0;
    n = n < p.num_tokens - start ? n : p.num_tokens - start;
    n = n > 0 ? n : 0;
    int64_t count = p.window > 0 && p.window < n ? p.window : n;
    const int64_t skip = n - count;
    count = count < p.max_count ? count : p.max_count;
    s.q0 = start + static_cast<int>(skip);
    s.count = static_cast<int>(count);
    const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block_size;
    int64_t c = p.context_lens[b];
    c = c > 0 ? c : 0;
    s.past = s.count > 0 ? static_cast<int>(c - given + skip) : 0;
    s.fresh = s.count > 0 ? static_cast<int>(c - given) : 0;
    c = c < cap ? c : cap;
    c = c < p.max_ctx ? c : p.max_ctx;
    s.ctx = s.count > 0 ? static_cast<int>(c) : 0;   // (no query tokens: nothing of the sequence is touched)
    s.stat0 = p.compact ? static_cast<int64_t>(b) * p.max_count : s.q0;
    return s;
}

// A row's weights are 2^((s - best) * scale) / sum of them, s its products q.k and `best` the one that weighs most, in
// both passes alike: the difference is taken first, where it is exact for those that weigh anything, so that scores of
// any size leave weights that add up to 1. (Maximum and logarithm of the sum in one number lost the sum, and the
// rounding of the scaled maximum, from scores of 2^12 on.)
// What the passes hand on: the maximum of s * sign(scale) and the sum; in the end (best, 1 / sum). A row that weighs
// nothing has an inverse of zero, one with a NaN that.
__device__ __forceinline__ float2 row_stats(const PrefillWeightsParams &p, float top, float sum) {
    if (sum == 0.f) return make_float2(0.f, 0.f);
    return make_float2(p.scale_log2 < 0.f ? -top : top, 1.f / sum);
}

// best * scale + log2(sum), so that 2^(s * scale - that) is the weight: half of row_stats to read, one instruction less
// a score. It rounds by 2^-19 at most up to this size, 1.3e-6 of the row's weights and no more than fp32 rounds a
// scaled score of that size by. NaN for larger ones (and rows with a NaN): they take the two numbers.
constexpr float kFoldedMost = 64.f;
__device__ __forceinline__ float folded_stats(const PrefillWeightsParams &p, float top, float sum) {
    if (sum == 0.f) return INFINITY;
    const float offset = fmaf(top, fabsf(p.scale_log2), log2f(sum));
    return fabsf(offset) <= kFoldedMost ? offset : __int_as_float(0x7fffffff);
}

// A row's statistics over one piece of its context; the only piece leaves the row's own.
__device__ __forceinline__ void leave_stats(const PrefillWeightsParams &p, int piece, int64_t stat, int head, float top,
                                            float sum) {
    if (p.nsplit == 1) p.rows[stat * p.num_heads + head] = row_stats(p, top, sum);   // (offsets: more pieces alone)
    else p.stats[(piece * p.stat_rows + stat) * p.num_heads + head] = make_float2(top, sum);
}

// The pieces' statistics of row i (of stat_rows x num_heads), put together.
__device__ __forceinline__ void merge_stats(const PrefillWeightsParams &p, int64_t i) {
    const int64_t all = p.stat_rows * p.num_heads;
    if (i >= all) return;
    const float size = fabsf(p.scale_log2);
    float top = -INFINITY, sum = 0.f;
    for (int s0 = 0; s0 < p.nsplit; s0 += 8) {
        float2 ml[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) ml[s] = s0 + s < p.nsplit ? p.stats[(s0 + s) * all + i] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float up = fmaxf(top, ml[s].x), ref = up == -INFINITY ? 0.f : up;
            sum = sum * fast_exp2((top - ref) * size) + ml[s].y * fast_exp2((ml[s].x - ref) * size);
            top = up;
        }
    }
    p.rows[i] = row_stats(p, top, sum);
    if (p.offsets) p.offsets[i] = folded_stats(p, top, sum);
}

struct EvictParams {
    const float *weights;         // [num_seqs, num_kv_heads, weights_stride]
    float *new_weights;           // [num_seqs, num_kv_heads, new_weights_stride]
    int32_t *kept;                // [num_seqs, num_kv_heads, kept_stride]
    int64_t weights_stride, new_weights_stride, kept_stride;
    void *k_cache, *v_cache;      // [num_blocks, block_size, num_kv_heads, row_bytes]
    const int32_t *block_tables;  // [num_seqs, max_blocks]
    const int32_t *new_tables;    // [num_seqs, max_new_blocks]
    const int32_t *context_lens, *keep_lens;
    int num_seqs, num_kv_heads, row_bytes, block_size, max_blocks, max_new_blocks, num_blocks;
    int max_ctx, max_keep;        // host bounds: what lies past them is cut
    int sinks, recent;
    int move_tokens;              // places a CTA fills (set by the launcher)
};

}  // namespace pa
