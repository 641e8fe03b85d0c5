// Arguments of the kernels that prepare and attend prompts: rotary positions
// (rope.cu) and several query tokens a sequence (prefill_*.cu).
#pragma once

#include <cfloat>

#include "device_common.cuh"

namespace pa {

// Rotary positions (rope.cu): heads of x rotated into out and, with
// num_kv_heads > 0, keys rotated and values copied into their cache slots.
struct RopeParams {
    const void *x;              // [num_tokens, num_heads, head_dim], token rows x_stride elements apart
    void *out;                  // the same, out_stride apart (may be x itself)
    const void *key, *value;    // [num_tokens, num_kv_heads, head_dim], or null with num_kv_heads 0
    void *k_cache, *v_cache;    // [num_slots, num_kv_heads, head_dim]
    const int64_t *slot_mapping;
    const int32_t *positions;   // [num_tokens]; negative: padding, nothing is written
    const double *inv_freq;     // [rotary_dim / 2] radians a position
    int64_t x_stride, out_stride, key_stride, value_stride;   // elements
    int64_t num_slots;
    int num_tokens, num_heads, num_kv_heads, head_dim, rotary_dim;
    int interleaved, transpose;
    float factor;               // multiplies cos and sin
    int tokens_per_cta, heads_per_cta;   // set by the launcher
};
constexpr int kRopeMaxHeadDim = 256;

// Attention of several query tokens a sequence (prefill_simt.cu, prefill_tc.cu).
// Query tokens are ragged: sequence b owns tokens query_start[b] ..
// query_start[b + 1] - 1. A row is one (query token, query head); the rows of
// one KV head are packed token by token, heads_per_tile heads each, into tiles.
struct PrefillParams {
    const void *query;            // [num_tokens, num_heads, head_dim]
    const void *k_cache, *v_cache;
    const int32_t *block_tables;  // null with contig_stride > 0
    const int32_t *context_lens;  // [num_seqs]
    const int32_t *query_start;   // [num_seqs + 1]
    void *out;                    // [num_tokens, num_heads, head_dim]
    float *part_out;              // split contexts: unmerged pieces (layout by kernel)
    float *part_max, *part_sum;
    int *status;
    int num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, group;
    int block_size, max_blocks, num_blocks;
    int contig_stride;            // > 0: contiguous [num_seqs, contig_stride, Hkv, D], no block table
    int max_query, max_ctx;       // host bounds: longer ones are cut
    int causal;                   // token i of q sees context - q + i + 1 tokens (else all)
    int out_type;                 // public dtype code
    int heads_per_tile, ntile;    // query heads of a KV head in one tile; tiles of the group
    int tile_tokens;              // query tokens in a row tile
    int nsplit;                   // prefill_simt: pieces a context is cut into; prefill_tc: 2 where the last
                                  //   wave's units may be cut, else 1
    int max_tail;                 // prefill_tc: units the cut wave can have
    int *tail_info;               // prefill_tc: its layout, prefill_rows: the tiles' prefix sums, for the merge
    int *counter;                 // prefill_tc: units drawn so far beyond one a CTA, or null (set to zero ahead)
    int *order;                   // prefill_tc: the sequences, longest context first, or null (batch order)
    int heads_per_cta;            // prefill_rows: KV heads (consumer warps) per CTA
    float scale_log2;
};

// Where a row's running maximum starts: finite, so that a row that has seen
// nothing keeps l = 0 with no inf - inf, and below every finite score but the
// lowest, which it equals.
constexpr float kLowestScore = -FLT_MAX;

// One sequence's extent, clamped so that no index leaves its array whatever
// the device-side lengths hold.
struct PrefillSeq {
    int q0, qlen;   // first query token, query tokens
    int ctx;        // context tokens
    int past;       // context tokens ahead of the first query token, of the lengths as given: what the
                    //   causal mask counts from, wherever the context is cut (negative: leading rows see nothing)
};

__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillParams &p, int b) {
    PrefillSeq s;
    s.q0 = p.query_start[b];
    const int64_t given = static_cast<int64_t>(p.query_start[b + 1]) - s.q0;
    int64_t n = given;
    if (s.q0 < 0 || s.q0 > p.num_tokens) n = 0;
    n = n < p.num_tokens - s.q0 ? n : p.num_tokens - s.q0;
    n = n < p.max_query ? n : p.max_query;
    s.qlen = n > 0 ? static_cast<int>(n) : 0;
    const int64_t cap = p.contig_stride > 0 ? p.contig_stride : static_cast<int64_t>(p.max_blocks) * p.block_size;
    int64_t c = p.context_lens[b];
    s.past = s.qlen > 0 ? static_cast<int>((c > 0 ? c : 0) - given) : 0;   // (given >= qlen >= 1: fits)
    c = c < cap ? c : cap;
    c = c < p.max_ctx ? c : p.max_ctx;
    s.ctx = c > 0 ? static_cast<int>(c) : 0;
    return s;
}

// Context tokens that query token i of a sequence sees.
__device__ __forceinline__ int prefill_sees(const PrefillParams &p, const PrefillSeq &s, int i) {
    if (!p.causal) return s.ctx;
    const int n = s.past + i + 1;
    return n < 0 ? 0 : n < s.ctx ? n : s.ctx;
}

// Warp-wide: the sequence that owns row tile `x` of the batch (its tiles
// enumerated sequence after sequence). Returns the sequence, or -1 past the
// last tile; `tile` is the index within the sequence.
__device__ __forceinline__ int prefill_find_tile(const PrefillParams &p, int x, int lane, int &tile) {
    int before = 0;
    for (int base = 0; base < p.num_seqs; base += 32) {
        const int b = base + lane;
        int n = 0;
        if (b < p.num_seqs) n = (prefill_seq(p, b).qlen + p.tile_tokens - 1) / p.tile_tokens;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, x < before + sum);
        if (hit) {
            const int l = __ffs(hit) - 1;
            tile = x - before - __shfl_sync(0xffffffffu, sum - n, l);
            return base + l;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return -1;
}

}  // namespace pa
