// Eviction from the paged cache by accumulated attention weight: of each
// sequence and KV head the first `sinks` tokens, the last `recent` and the
// heaviest others stay, in their order, moved together into other blocks.
//
// Two kernels.
//  * Choice, one CTA a (sequence, KV head). Weights become unsigned keys that sort
//    alike; a bitwise search from the top bit finds the k-th largest key (bit set
//    where k keys or more reach it: one count over the CTA a bit). The keys stay in
//    registers where the context has 32,768 tokens or less (32 a thread), else they
//    are read again for each bit; once few enough share the bits found, those alone
//    are searched on, from shared memory. Keys above the threshold are taken, and of
//    those equal to it the first ones; ranks come from ballots and one scan over the
//    warps, so positions leave in order without a sort and without atomics that
//    would show in the result.
//    Bound: the latency of 32 counts (a barrier each) and of two reads of the weights.
//  * Move: rows of 16-byte vectors, all heads of a kept place together, because a
//    place's heads are contiguous where they go (they come from different tokens). Each
//    element is read once and written once, so HBM is the bound.
#include <algorithm>

#include "internal.h"
#include "weights_common.cuh"

namespace pa {

namespace {

constexpr int kChooseThreads = 1024;
constexpr int kChooseWarps = kChooseThreads / 32;
constexpr int kChooseKeys = 32;      // keys a thread, at most, that stay in registers
constexpr int kListKeys = 2;         // keys a thread of the short list
constexpr int kList = kListKeys * kChooseThreads;
constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 32;      // places a CTA fills
constexpr int kMoveHeads = 16;       //   of this many heads, at most
constexpr int kMoveUnroll = 4;       // vectors of K and of V a thread has in flight

struct EvictSeq {
    int len;      // context tokens
    int keep;     // tokens that stay (-1: the sequence is left alone)
    int sinks, recent;
};

__device__ __forceinline__ EvictSeq evict_seq(const EvictParams &p, int b) {
    EvictSeq s;
    const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block_size;
    int64_t n = p.context_lens[b];
    n = n < p.max_ctx ? n : p.max_ctx;
    n = n < cap ? n : cap;
    s.len = n > 0 ? static_cast<int>(n) : 0;
    const int keep = p.keep_lens[b];
    s.keep = keep < 0 ? -1 : min(min(keep, p.max_keep), s.len);
    s.recent = min(p.recent, max(s.keep, 0));
    s.sinks = min(p.sinks, max(s.keep, 0) - s.recent);
    return s;
}

// An unsigned key that sorts as the weight does; NaN counts as minus infinity, and
// zeros of both signs as one. Never 0, which stands for no candidate.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The CTA's sum of one count a warp lane; `turn` alternates so that one barrier a sum suffices.
__device__ __forceinline__ int cta_sum(int x, int (*part)[kChooseWarps], int turn) {
    x = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, part[turn][threadIdx.x & 31]);
}

// Each warp owns the positions warp * keys * 32 + i * 32 + lane of a chunk, i < kKeys; with kResident
// one chunk is the whole context, else the chunks follow one another.
template <int kKeys, bool kResident>
__global__ void __launch_bounds__(kChooseThreads, 1)
evict_choose_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int part[2][kChooseWarps];
    __shared__ int above[kChooseWarps], equal[kChooseWarps];
    __shared__ uint32_t list[kList];
    __shared__ int listed;
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.x / p.num_kv_heads, h = blockIdx.x % p.num_kv_heads;
    const EvictSeq s = evict_seq(p, b);
    if (s.keep <= 0) return;
    const int64_t row = static_cast<int64_t>(b) * p.num_kv_heads + h;
    const float *w = p.weights + row * p.weights_stride;
    float *new_w = p.new_weights + row * p.new_weights_stride;
    int32_t *kept = p.kept + row * p.kept_stride;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (s.keep == s.len) {   // everything stays
        for (int t = threadIdx.x; t < s.len; t += kChooseThreads) {
            kept[t] = t;
            new_w[t] = w[t];
        }
        return;
    }
    constexpr int kChunk = kKeys * kChooseThreads;
    const int chunks = kResident ? 1 : (s.len + kChunk - 1) / kChunk;
    const int first = s.sinks, last = s.len - s.recent;   // the candidates
    const int want = s.keep - s.sinks - s.recent;         // how many of them stay
    auto place = [&](int chunk, int i) { return chunk * kChunk + (warp * kKeys + i) * 32 + lane; };
    auto key_at = [&](int t) -> uint32_t { return t >= first && t < last ? weight_key(w[t]) : 0u; };

    uint32_t key[kKeys];
    auto load = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) key[i] = key_at(place(chunk, i));
    };
    if (kResident) load(0);

    // threshold: the want-th largest key; over: how many keys are larger
    uint32_t threshold = 0;
    int over = 0, reach = last - first, turn = 0, bit = 31;
    if (threadIdx.x == 0) listed = 0;
    if (want > 0) {
        for (; bit >= 0 && reach - over > kList; --bit) {
            const uint32_t probe = threshold | (1u << bit);
            int n = 0;
            for (int c = 0; c < chunks; ++c) {
                if (!kResident) load(c);
#pragma unroll
                for (int i = 0; i < kKeys; ++i) n += key[i] >= probe;
            }
            n = cta_sum(n, part, turn);
            turn ^= 1;
            if (n >= want) {
                threshold = probe;
                reach = n;
            } else {
                over = n;
            }
        }
        // the few keys that share the bits found so far
        if (bit >= 0) {
            __syncthreads();   // (listed is zero)
            const uint32_t found = bit == 31 ? 0u : ~((2u << bit) - 1u);   // the mask of those bits
            for (int c = 0; c < chunks; ++c) {
                if (!kResident) load(c);
#pragma unroll
                for (int i = 0; i < kKeys; ++i) {
                    const bool in = key[i] != 0u && (key[i] & found) == threshold;
                    const unsigned votes = __ballot_sync(0xffffffffu, in);
                    if (votes == 0u) continue;
                    int at = 0;
                    if (lane == 0) at = atomicAdd(&listed, __popc(votes));   // (their order does not matter)
                    at = __shfl_sync(0xffffffffu, at, 0) + __popc(votes & ((1u << lane) - 1u));
                    if (in) list[at] = key[i];
                }
            }
            __syncthreads();
            uint32_t mine[kListKeys];
#pragma unroll
            for (int i = 0; i < kListKeys; ++i) {
                const int at = threadIdx.x + i * kChooseThreads;
                mine[i] = at < listed ? list[at] : 0u;
            }
            const int fixed = over;   // keys above all of the list
            for (; bit >= 0; --bit) {
                const uint32_t probe = threshold | (1u << bit);
                int n = 0;
#pragma unroll
                for (int i = 0; i < kListKeys; ++i) n += mine[i] >= probe;
                n = fixed + cta_sum(n, part, turn);
                turn ^= 1;
                if (n >= want) threshold = probe;
                else over = n;
            }
        }
    } else {
        threshold = 0xffffffffu;   // (no weight has this key)
    }
    const int want_equal = max(want - over, 0);   // of the keys equal to the threshold, the first so many

    // ranks: kept so far, equal keys so far, of the warps and chunks before
    int kept_before = 0, equal_before = 0;
    for (int c = 0; c < chunks; ++c) {
        if (!kResident) load(c);
        int n_above = 0, n_equal = 0;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int t = place(c, i);
            const bool forced = t < first || (t >= last && t < s.len);
            n_above += __popc(__ballot_sync(0xffffffffu, forced || key[i] > threshold));
            n_equal += __popc(__ballot_sync(0xffffffffu, key[i] == threshold));
        }
        __syncthreads();   // (the chunk before has been read)
        if (lane == 0) {
            above[warp] = n_above;
            equal[warp] = n_equal;
        }
        __syncthreads();
        // equal keys of the warps before, then what those warps keep
        int eq = equal[lane], eq_scan = eq;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, eq_scan, d);
            if (lane >= d) eq_scan += o;
        }
        const int eq_first = equal_before + eq_scan - eq;
        int keeps = above[lane] + min(max(want_equal - eq_first, 0), eq), keeps_scan = keeps;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, keeps_scan, d);
            if (lane >= d) keeps_scan += o;
        }
        int at = kept_before + __shfl_sync(0xffffffffu, keeps_scan - keeps, warp);
        int eq_at = __shfl_sync(0xffffffffu, eq_first, warp);
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int t = place(c, i);
            const bool same = key[i] == threshold;
            const unsigned below = (1u << lane) - 1u;
            const unsigned same_votes = __ballot_sync(0xffffffffu, same);
            const bool stays = t < first || (t >= last && t < s.len) || key[i] > threshold ||
                               (same && eq_at + __popc(same_votes & below) < want_equal);
            const unsigned votes = __ballot_sync(0xffffffffu, stays);
            if (stays) {
                const int to = at + __popc(votes & below);
                kept[to] = t;
                new_w[to] = w[t];
            }
            at += __popc(votes);
            eq_at += __popc(same_votes);
        }
        kept_before += __shfl_sync(0xffffffffu, keeps_scan, 31);
        equal_before += __shfl_sync(0xffffffffu, eq_scan, 31);
    }
}

__device__ __forceinline__ uint4 load_row(const uint4 *p) { return __ldcs(p); }

// One CTA: kMoveTokens places of one sequence, up to kMoveHeads heads of each.
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int64_t from[kMoveTokens * kMoveHeads];   // (place, head): byte offset of its row, or -1
    __shared__ int64_t to[kMoveTokens];                  // place: byte offset of its token's first head
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.y;
    const EvictSeq s = evict_seq(p, b);
    const int j0 = blockIdx.x * kMoveTokens;
    const int places = min(kMoveTokens, s.keep - j0);
    if (places <= 0) return;
    const int head0 = blockIdx.z * kMoveHeads;
    const int heads = min(kMoveHeads, p.num_kv_heads - head0);
    const int64_t token_bytes = static_cast<int64_t>(p.num_kv_heads) * p.row_bytes;
    const int32_t *table = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
    const int32_t *new_table = p.new_tables + static_cast<int64_t>(b) * p.max_new_blocks;
    // byte offset of a token of the pool (a block outside the pool: -1)
    auto token_at = [&](const int32_t *tab, int t) -> int64_t {
        const int blk = tab[t / p.block_size];
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) return -1;
        return (static_cast<int64_t>(blk) * p.block_size + t % p.block_size) * token_bytes;
    };
    for (int i = threadIdx.x; i < kMoveTokens * heads; i += kMoveThreads) {
        const int j = i % kMoveTokens, h = i / kMoveTokens;
        if (j >= places) continue;
        const int t = p.kept[(static_cast<int64_t>(b) * p.num_kv_heads + head0 + h) * p.kept_stride + j0 + j];
        const int64_t at = token_at(table, t);
        from[j * heads + h] = at < 0 ? -1 : at + static_cast<int64_t>(head0 + h) * p.row_bytes;
    }
    if (threadIdx.x < places) to[threadIdx.x] = token_at(new_table, j0 + threadIdx.x);
    __syncthreads();

    const int vecs = p.row_bytes / 16;
    const int total = places * heads * vecs;
    const unsigned char *k = static_cast<const unsigned char *>(p.k_cache), *v = static_cast<const unsigned char *>(p.v_cache);
    for (int i0 = threadIdx.x; i0 < total; i0 += kMoveThreads * kMoveUnroll) {
        uint4 kv[kMoveUnroll], vv[kMoveUnroll];
        int64_t dst[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int i = i0 + u * kMoveThreads;
            dst[u] = -1;
            if (i >= total) continue;
            const int r = i / vecs, c = i - r * vecs;   // row (place, head), vector
            const int j = r / heads;
            const int64_t src = from[r];
            if (src < 0 || to[j] < 0) continue;
            dst[u] = to[j] + static_cast<int64_t>(head0 + r - j * heads) * p.row_bytes + c * 16;
            kv[u] = load_row(reinterpret_cast<const uint4 *>(k + src + c * 16));
            vv[u] = load_row(reinterpret_cast<const uint4 *>(v + src + c * 16));
        }
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            if (dst[u] < 0) continue;
            *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(p.k_cache) + dst[u]) = kv[u];
            *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(p.v_cache) + dst[u]) = vv[u];
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t stream) {
    const dim3 rows(static_cast<unsigned>(p.num_seqs * p.num_kv_heads));
    cudaError_t e;
    if (p.max_ctx <= kChooseThreads)
        e = launch_kernel(evict_choose_kernel<1, true>, rows, dim3(kChooseThreads), 0, stream, 1u, p);
    else if (p.max_ctx <= 8 * kChooseThreads)
        e = launch_kernel(evict_choose_kernel<8, true>, rows, dim3(kChooseThreads), 0, stream, 1u, p);
    else if (p.max_ctx <= kChooseKeys * kChooseThreads)
        e = launch_kernel(evict_choose_kernel<kChooseKeys, true>, rows, dim3(kChooseThreads), 0, stream, 1u, p);
    else
        e = launch_kernel(evict_choose_kernel<kChooseKeys, false>, rows, dim3(kChooseThreads), 0, stream, 1u, p);
    if (e != cudaSuccess) return e;
    const int most = std::min(p.max_keep, p.max_ctx);
    const dim3 grid(static_cast<unsigned>((most + kMoveTokens - 1) / kMoveTokens), static_cast<unsigned>(p.num_seqs),
                    static_cast<unsigned>((p.num_kv_heads + kMoveHeads - 1) / kMoveHeads));
    return launch_kernel(evict_move_kernel, grid, dim3(kMoveThreads), 0, stream, 1u, p);
}

}  // namespace pa
