// Eviction from the paged cache by accumulated attention weight: of each
// sequence and KV head the first `sinks` tokens, the last `recent` and the
// heaviest others stay, in their order, moved together into other blocks.
//
// Two kernels.
//  * Choice, a CTA or a cluster of them a (sequence, KV head). Weights become unsigned keys
//    that sort alike; the k-th largest is found digit by digit (8 bits, from the top): a
//    histogram of the keys that share the digits found so far, and the bin in which the
//    k-th falls. Four rounds, each a pass over keys in registers (16 a thread; contexts
//    past 64 K are read again), three barriers, and in a cluster one exchange of 256 totals
//    through distributed shared memory. Eight copies of the histogram, by lane: weights
//    of one sign and few exponents fall into few bins. Keys above the threshold are
//    taken, and of those equal to it the first ones; ranks come from ballots and one scan
//    over the warps, so positions leave in order without a sort and without atomics
//    that would show in the result. Bound: the latency of those rounds. (Found bit by
//    bit, a count over 1,024 threads each, the whole call took 60.7 us for 16 sequences
//    of 4,164 tokens, now 55.0, and 37 for one of 32,768, now 18.7.)
//  * Move: rows of 16-byte vectors, all heads of a kept place together, because a
//    place's heads are contiguous where they go (they come from different tokens). Each
//    element is read once and written once, so HBM is the bound: 268 MB in 41 us
//    (0.98 of the copy rate; the choice of that call takes 11.7 us, that of 8 heads of one
//    context of 32,768 tokens 15.4).
#include <algorithm>

#include "internal.h"
#include "weights_common.cuh"

namespace pa {

namespace {

constexpr int kChooseThreads = 512;
constexpr int kChooseWarps = kChooseThreads / 32;
constexpr int kChooseKeys = 16;      // keys a thread holds
constexpr int kChooseChunk = kChooseKeys * kChooseThreads;
constexpr int kBins = 256, kCopies = 8;
constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 32;      // places a CTA fills, at most
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

// (not volatile: several are on their way at once)
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// CTA r of a cluster of c owns every chunk n with n % c == r of chunks of kKeys x 512 positions, and a warp of it
// the positions warp * kKeys * 32 + i * 32 + lane of a chunk, i < kKeys. kResident: one chunk a CTA.
template <int kKeys, bool kResident>
__global__ void __launch_bounds__(kChooseThreads, 1)
evict_choose_kernel(const __grid_constant__ EvictParams p, const int cluster) {
    __shared__ __align__(16) int bins[kBins * kCopies];   // [bin][copy]
    __shared__ int totals[2][kBins];                      // this CTA's, by the parity of the round
    __shared__ int s_digit, s_over, s_scan[kBins / 32];
    __shared__ int above[kChooseWarps], equal[kChooseWarps];
    __shared__ int2 s_counts[2];                          // (kept without equals, equals) of this CTA's chunk
    grid_dependency_wait();
    grid_dependents_launch();
    const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int unit = blockIdx.x / cluster;
    const int b = unit / p.num_kv_heads, h = unit % p.num_kv_heads;
    const EvictSeq s = evict_seq(p, b);
    if (s.keep <= 0) return;   // (every CTA of the cluster alike)
    const int64_t row = static_cast<int64_t>(b) * p.num_kv_heads + h;
    const float *w = p.weights + row * p.weights_stride;
    float *new_w = p.new_weights + row * p.new_weights_stride;
    int32_t *kept = p.kept + row * p.kept_stride;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (s.keep == s.len) {   // everything stays
        for (int t = rank * kChooseThreads + threadIdx.x; t < s.len; t += cluster * kChooseThreads) {
            kept[t] = t;
            new_w[t] = w[t];
        }
        return;
    }
    constexpr int kChunk = kKeys * kChooseThreads;
    const int all_chunks = (s.len + kChunk - 1) / kChunk;
    const int rounds = kResident ? 1 : (all_chunks + cluster - 1) / cluster;   // chunks a CTA goes through
    const int first = s.sinks, last = s.len - s.recent;   // the candidates
    int want = s.keep - s.sinks - s.recent;               // how many of them stay
    auto place = [&](int round, int i) { return (round * cluster + rank) * kChunk + (warp * kKeys + i) * 32 + lane; };
    uint32_t key[kKeys];
    float val[kKeys];
    auto load = [&](int round) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) val[i] = place(round, i) < s.len ? w[place(round, i)] : 0.f;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int t = place(round, i);
            key[i] = t >= first && t < last ? weight_key(val[i]) : 0u;
        }
    };
    if (kResident) load(0);
    for (int i = threadIdx.x; i < kBins * kCopies; i += kChooseThreads) bins[i] = 0;

    // threshold: the want-th largest key. A round fixes the next digit of it; want counts on within the keys that
    // share the digits so far.
    uint32_t threshold = 0;
    if (want > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            const uint32_t found = shift == 24 ? 0u : ~0u << (shift + 8);   // the bits fixed so far
            __syncthreads();   // (the histogram is empty)
            for (int c = 0; c < rounds; ++c) {
                if (!kResident) load(c);
#pragma unroll
                for (int i = 0; i < kKeys; ++i)
                    if (key[i] != 0u && (key[i] & found) == threshold)
                        atomicAdd(&bins[((key[i] >> shift) & 255u) * kCopies + (lane & (kCopies - 1))], 1);
            }
            __syncthreads();
            // thread t: bin 255 - t, the largest digits first
            int count = 0, upto = 0;
            const int bin = kBins - 1 - static_cast<int>(threadIdx.x);
            if (threadIdx.x < kBins) {
                int4 *const at = reinterpret_cast<int4 *>(bins) + 2 * bin;
                const int4 x = at[0], y = at[1];
                count = x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w;
                at[0] = at[1] = make_int4(0, 0, 0, 0);   // for the next round
            }
            if (cluster > 1) {
                int *const total = totals[(shift >> 3) & 1];
                if (threadIdx.x < kBins) total[bin] = count;
                cluster_sync_all();
                if (threadIdx.x < kBins) {
                    int n[kMaxClusterSplits];
#pragma unroll
                    for (int r = 0; r < kMaxClusterSplits; ++r)
                        n[r] = r < cluster ? ld_cluster_s32(cluster_map(smem_addr(&total[bin]), r)) : 0;
                    count = 0;
#pragma unroll
                    for (int r = 0; r < kMaxClusterSplits; ++r) count += n[r];
                }
            }
            if (threadIdx.x < kBins) {
                upto = count;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int o = __shfl_up_sync(0xffffffffu, upto, d);
                    if (lane >= d) upto += o;
                }
                if (lane == 31) s_scan[warp] = upto;
            }
            __syncthreads();
            if (threadIdx.x < kBins) {
#pragma unroll
                for (int i = 0; i < kBins / 32; ++i) upto += i < warp ? s_scan[i] : 0;
                if (upto - count < want && upto >= want) {   // upto - count keys have a larger digit
                    s_digit = bin;
                    s_over = upto - count;
                }
            }
            __syncthreads();
            threshold |= static_cast<uint32_t>(s_digit) << shift;
            want -= s_over;
        }
    } else {
        threshold = 0xffffffffu;   // (no weight has this key)
    }
    const int want_equal = max(want, 0);   // of the keys equal to the threshold, the first so many

    // ranks: kept so far, equal keys so far, of the warps and chunks before
    int kept_before = 0, equal_before = 0;
    for (int c = 0; c < rounds; ++c) {
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
        if (cluster > 1) {   // the chunks of the CTAs before, and after, in this round
            if (warp == 0) {
                const int a = __reduce_add_sync(0xffffffffu, lane < kChooseWarps ? above[lane] : 0);
                const int e = __reduce_add_sync(0xffffffffu, lane < kChooseWarps ? equal[lane] : 0);
                if (lane == 0) s_counts[c & 1] = make_int2(a, e);
            }
            cluster_sync_all();
        }
        int others_kept = 0, others_equal = 0, all_kept = 0, all_equal = 0;
        if (cluster > 1) {
            for (int r = 0; r < cluster; ++r) {
                const uint32_t at = cluster_map(smem_addr(&s_counts[c & 1]), r);
                const int a = ld_cluster_s32(at), e = ld_cluster_s32(at + 4);
                const int keeps = a + min(max(want_equal - equal_before - all_equal, 0), e);
                if (r < rank) {
                    others_kept += keeps;
                    others_equal += e;
                }
                all_kept += keeps;
                all_equal += e;
            }
        }
        // equal keys of the warps before, then what those warps keep
        const int eq = lane < kChooseWarps ? equal[lane] : 0;
        int eq_scan = eq;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, eq_scan, d);
            if (lane >= d) eq_scan += o;
        }
        const int eq_first = equal_before + others_equal + eq_scan - eq;
        const int keeps = (lane < kChooseWarps ? above[lane] : 0) + min(max(want_equal - eq_first, 0), eq);
        int keeps_scan = keeps;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, keeps_scan, d);
            if (lane >= d) keeps_scan += o;
        }
        int at = kept_before + others_kept + __shfl_sync(0xffffffffu, keeps_scan - keeps, warp);
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
                new_w[to] = val[i];
            }
            at += __popc(votes);
            eq_at += __popc(same_votes);
        }
        kept_before += cluster > 1 ? all_kept : __shfl_sync(0xffffffffu, keeps_scan, 31);
        equal_before += cluster > 1 ? all_equal : __shfl_sync(0xffffffffu, eq_scan, 31);
    }
    if (cluster > 1) cluster_sync_all();   // the peers have read this CTA's counts
}

__device__ __forceinline__ uint4 load_row(const uint4 *p) { return __ldcs(p); }

// One CTA: p.move_tokens places of one sequence, up to kMoveHeads heads of each.
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int64_t from[kMoveTokens * kMoveHeads];   // (place, head): byte offset of its row, or -1
    __shared__ int64_t to[kMoveTokens];                  // place: byte offset of its token's first head
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.y;
    const EvictSeq s = evict_seq(p, b);
    const int j0 = blockIdx.x * p.move_tokens;
    const int places = min(p.move_tokens, s.keep - j0);
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
    for (int i = threadIdx.x; i < places * heads; i += kMoveThreads) {
        const int h = i / places, j = i - h * places;
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

cudaError_t launch_evict(EvictParams &p, int sms, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads;
    const int chunks = (p.max_ctx - 1) / kChooseChunk + 1;
    // a cluster where one CTA's registers do not hold the context
    int cluster = 1;
    while (cluster < kMaxClusterSplits && cluster < chunks) cluster *= 2;
    cudaError_t e;
    if (p.max_ctx <= 2 * kChooseThreads)
        e = launch_kernel(evict_choose_kernel<2, true>, dim3(static_cast<unsigned>(rows)), dim3(kChooseThreads), 0, stream, 1u, p, 1);
    else
        e = launch_kernel(chunks <= cluster ? evict_choose_kernel<kChooseKeys, true> : evict_choose_kernel<kChooseKeys, false>,
                          dim3(static_cast<unsigned>(rows * cluster)), dim3(kChooseThreads), 0, stream, static_cast<unsigned>(cluster), p,
                          cluster);
    if (e != cudaSuccess) return e;
    const int64_t most = std::min(p.max_keep, p.max_ctx);
    const unsigned groups = static_cast<unsigned>((p.num_kv_heads + kMoveHeads - 1) / kMoveHeads);
    // few places: fewer a CTA, so that all SMs have some (4,096 places of 8 heads of 128: 12.6 us at 32, 10.7 at 8)
    p.move_tokens = kMoveTokens;
    while (p.move_tokens > 8 && (most + p.move_tokens - 1) / p.move_tokens * p.num_seqs * groups < 3 * static_cast<int64_t>(sms))
        p.move_tokens /= 2;
    const dim3 grid(static_cast<unsigned>((most + p.move_tokens - 1) / p.move_tokens), static_cast<unsigned>(p.num_seqs), groups);
    return launch_kernel(evict_move_kernel, grid, dim3(kMoveThreads), 0, stream, 1u, p);
}

}  // namespace pa
