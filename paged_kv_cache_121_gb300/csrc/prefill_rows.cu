// Attention of a few query tokens a sequence -- drafts to verify, single
// decoder tokens against an encoder's states -- where a KV head has at most 16
// rows (query tokens x the query heads that share it), 16-bit caches in blocks
// of 16 to 256 tokens or contiguous.
//
// Bound: the cache's bytes. With 16 rows to a K/V row the products are a
// quarter of what mma.sync does at full HBM rate, and S, P and O stay in one
// warp's registers; padded to the 128 rows of a tcgen05 tile they would make a
// chain of waits a tile instead. Measured on GB300, prefill_tc against this with
// its merge: 16 sequences x 4 tokens over 4,164-token contexts, 32 / 8 heads of
// 128, 57.8 -> 52.5 us (274 MB: 5.2 TB/s, 0.77 of the copy rate); 64 single tokens
// over 200-1,500 states, 16 heads of 64, 63.6 -> 42 (212 MB: 5.0 TB/s, 0.74).
//
// A CTA (one per SM) holds up to 8 KV heads, a consumer warp each, and a
// producer warp that streams 16-token tiles of all of them, one TMA box of K
// and one of V, through an mbarrier ring. For one group of KV heads the batch's
// tiles are laid end to end, sequence after sequence, and cut into equal ranges
// per CTA on the device, where the lengths are: every CTA gets the same bytes
// however ragged the batch. A CTA's first and last segment may be pieces of a
// sequence: they go to the workspace, slots 2 c and 2 c + 1 of CTA c, and the
// merge joins them; sequences held whole are written by their CTA.
#include "internal.h"
#include "mma_tile.cuh"
#include "prompt_common.cuh"

namespace pa {

namespace {

constexpr int kTT = 16;                 // tokens per tile
constexpr int kMaxHeads = 8;            // consumer warps
constexpr int kMaxStages = 16;
constexpr int kRingBytes = 192 * 1024;  // three stages of 8 heads of 128, six of 64

// The tiles a sequence takes: none without query tokens, one at least with any
// (an empty context still has rows of zeros to write).
__device__ __forceinline__ int seq_tiles(const PrefillParams &p, const PrefillSeq &s) {
    if (s.qlen == 0) return 0;
    return max(1, (prefill_sees(p, s, s.qlen - 1) + kTT - 1) / kTT);
}

// P[b] = tiles of sequences 0 .. b - 1, P[B] = all of them, and ctx[b]. All threads.
__device__ void rows_prefix(const PrefillParams &p, int *P, int *ctx, int *scratch) {
    const int B = p.num_seqs, nt = blockDim.x;
    const int per = (B + nt - 1) / nt, b0 = static_cast<int>(threadIdx.x) * per;
    int sum = 0;
    for (int b = b0; b < min(B, b0 + per); ++b) {
        const PrefillSeq s = prefill_seq(p, b);
        ctx[b] = s.ctx;
        P[b] = seq_tiles(p, s);   // (its count, until the sums are known)
        sum += P[b];
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += scratch[w];
    for (int b = b0; b < min(B, b0 + per); ++b) {
        const int n = P[b];
        P[b] = run;
        run += n;
    }
    if (threadIdx.x == static_cast<unsigned>(nt - 1)) P[B] = run;   // the last thread's running sum is the total
    __syncthreads();
}

// The sequence that owns tile g: the largest b with P[b] <= g.
__device__ __forceinline__ int rows_seq_of(const int *P, int B, int g) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P[mid] <= g) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// W tiles over C CTAs (C <= W): the first W % C take one more.
__device__ __forceinline__ int rows_begin(int c, int W, int C) { return c * (W / C) + min(c, W % C); }
__device__ __forceinline__ int rows_owner(int x, int W, int C) {
    const int q = W / C, more = W % C, edge = more * (q + 1);
    return x < edge ? x / (q + 1) : more + (x - edge) / q;
}

// Workspace row of (slot, KV head, row): 16 rows a KV head.
__device__ __forceinline__ int64_t piece_row(const PrefillParams &p, int slot, int kvh, int r) {
    return (static_cast<int64_t>(slot) * p.num_kv_heads + kvh) * 16 + r;
}

template <int D>
__device__ __forceinline__ void rows_epilogue(const PrefillParams &p, const WarpState<D> &st, const PrefillSeq &s,
                                              int kvh, int slot, int lane) {
    const int q4 = lane & 3, rows = s.qlen * p.group;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = (lane >> 2) + 8 * half;
        if (r >= rows) continue;
        const float m = half ? st.m1 : st.m0, l = half ? st.l1 : st.l0;
        if (slot < 0) {
            const float inv = l > 0.f ? 1.f / l : l;   // 0: a row that sees nothing; NaN stays NaN
            const int t = r / p.group;
            const int64_t row = static_cast<int64_t>(s.q0 + t) * p.num_heads + kvh * p.group + (r - t * p.group);
#pragma unroll
            for (int dn = 0; dn < D / 8; ++dn)
                store_pair_as(p.out, p.out_type, row * D + 8 * dn + 2 * q4, st.o[dn][2 * half] * inv,
                              st.o[dn][2 * half + 1] * inv);
        } else {                                       // a piece: unnormalised, with its maximum and sum
            const int64_t row = piece_row(p, slot, kvh, r);
#pragma unroll
            for (int dn = 0; dn < D / 8; ++dn)
                *reinterpret_cast<float2 *>(p.part_out + row * D + 8 * dn + 2 * q4) =
                    make_float2(st.o[dn][2 * half], st.o[dn][2 * half + 1]);
            if (q4 == 0) {
                p.part_max[row] = m;
                p.part_sum[row] = l;
            }
        }
    }
}

template <int D, bool kF16>
__global__ void __launch_bounds__(32 * (kMaxHeads + 1), 1)
prefill_rows_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                    const __grid_constant__ PrefillParams p) {
    constexpr int kHalves = D / 64;
    constexpr int kHalfStride = kTT * 128;               // one 64-dim half of one head's tile
    constexpr int kHeadStride = kHalves * kHalfStride;   // one head's K (or V) rows of a tile
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int hpc = p.heads_per_cta;
    const int stage_bytes = 2 * hpc * kTT * D * 2;
    const int nstages = min(kRingBytes / stage_bytes, kMaxStages);
    const int v_off = stage_bytes / 2;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kRingBytes);   // full[kMaxStages], empty[kMaxStages]
    int *P = reinterpret_cast<int *>(bars + 2 * kMaxStages);            // [num_seqs + 1]
    int *ctx = P + p.num_seqs + 1;                                      // [num_seqs]
    __shared__ int s_scratch[32];
    __shared__ int s_abort;
    __shared__ int s_issued;

    const int c = blockIdx.x, B = p.num_seqs, hgrp = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        for (int s = 0; s < nstages; ++s) {
            mbar_init(smem_addr(&bars[s]), 1);
            mbar_init(smem_addr(&bars[kMaxStages + s]), hpc);
        }
        s_abort = 0;
        s_issued = 0;
        mbar_fence_init();
    }
    grid_dependency_wait();
    rows_prefix(p, P, ctx, s_scratch);
    const int W = P[B];
    if (c == 0 && hgrp == 0)   // for the merge
        for (int i = threadIdx.x; i <= B; i += blockDim.x) p.tail_info[i] = P[i];
    const int C = min(static_cast<int>(gridDim.x), W);   // no range is empty
    if (c >= C) return;
    const int start = rows_begin(c, W, C), end = rows_begin(c + 1, W, C);
    const int ntiles = end - start;
    const bool contig = p.contig_stride > 0;

    if (warp == hpc) {
        // ------------------------------ producer ------------------------------
        // Lane l holds block, token coordinate and fill of tile start + 32 k + l
        // of the current chunk k, the next chunk fetched ahead.
        const uint64_t policy = l2_policy_evict_first();
        auto lookup = [&](int i, int &blk, int &off) {
            blk = 0;
            off = -1;   // nothing to load
            if (i < ntiles) {
                const int g = start + i, b = rows_seq_of(P, B, g), tok = (g - P[b]) * kTT;
                if (tok < ctx[b]) {
                    if (contig) {
                        off = b * p.contig_stride + tok;
                    } else {
                        blk = p.block_tables[static_cast<int64_t>(b) * p.max_blocks + tok / p.block_size];
                        off = tok % p.block_size;
                    }
                }
            }
        };
        const int head0 = hgrp * hpc;
        int cur_blk, cur_off, nxt_blk, nxt_off;
        lookup(lane, cur_blk, cur_off);
        lookup(32 + lane, nxt_blk, nxt_off);
        int issued = 0;
        for (int i = 0; i < ntiles; ++i) {
            if ((i & 31) == 0 && i > 0) {
                cur_blk = nxt_blk;
                cur_off = nxt_off;
                lookup(i + 32 + lane, nxt_blk, nxt_off);
            }
            const int blk = __shfl_sync(0xffffffffu, cur_blk, i & 31), off = __shfl_sync(0xffffffffu, cur_off, i & 31);
            int ok = 1;
            if (lane == 0) {
                const int s = i % nstages, k = i / nstages;
                if (k > 0) {
                    if (*reinterpret_cast<volatile int *>(&s_abort)) {
                        ok = 0;
                    } else if (!mbar_wait(smem_addr(&bars[kMaxStages + s]), (k - 1) & 1)) {
                        record_status(p.status, kStatusTimeout);
                        s_abort = 1;
                        ok = 0;
                    }
                }
                if (ok) {
                    const uint32_t full = smem_addr(&bars[s]), kdst = smem_addr(smem + s * stage_bytes);
                    if (off < 0) {
                        mbar_arrive(full);
                    } else {
                        mbar_arrive_expect_tx(full, static_cast<uint32_t>(stage_bytes));
                        // (dim, token, half, head, block), innermost first
                        tma_load_5d(kdst, &tmap_k, 0, off, 0, head0, blk, full, policy);
                        tma_load_5d(kdst + v_off, &tmap_v, 0, off, 0, head0, blk, full, policy);
                    }
                    issued = i + 1;
                }
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        }
        if (lane == 0) s_issued = issued;
    } else if (warp < hpc) {
        // ------------------------------ consumers -----------------------------
        const int kvh = hgrp * hpc + warp, r = lane >> 2;
        const float sl2 = p.scale_log2;
        auto tok_off = [](int t) -> int { return t * 128; };
        const uint16_t *query = static_cast<const uint16_t *>(p.query);
        // the query row of tile row i (token i / group, head i % group)
        auto query_row = [&](const PrefillSeq &s, int i) {
            const int t = i / p.group;
            return query + (static_cast<int64_t>(s.q0 + t) * p.num_heads + kvh * p.group + (i - t * p.group)) * D;
        };
        WarpState<D> st;
        uint32_t qa[D / 16][4];
        int b = rows_seq_of(P, B, start), seg_end = 0, sees0 = 0, sees1 = 0;
        PrefillSeq s = prefill_seq(p, b), next = s;
        bool open = false;
        auto close = [&]() {   // the segment of sequence b is done
            st.reduce_sums();
            const bool whole = P[b] >= start && seg_end <= end;
            rows_epilogue<D>(p, st, s, kvh, whole ? -1 : 2 * c + (start >= P[b] ? 0 : 1), lane);
        };
        bool ok = true;
        for (int i = 0; i < ntiles; ++i) {
            const int g = start + i;
            if (!open || g >= seg_end) {
                if (open) {
                    close();
                    while (P[b + 1] <= g) ++b;   // skips sequences without tiles
                    s = next;
                }
                open = true;
                seg_end = P[b + 1];
                const int rows = s.qlen * p.group;
                load_query_fragments<D>(qa, reinterpret_cast<const uint32_t *>(query_row(s, r)),
                                        reinterpret_cast<const uint32_t *>(query_row(s, r + 8)), r < rows, r + 8 < rows,
                                        lane);
                sees0 = r < rows ? prefill_sees(p, s, r / p.group) : 0;
                sees1 = r + 8 < rows ? prefill_sees(p, s, (r + 8) / p.group) : 0;
                st.init();
                st.m0 = st.m1 = kLowestScore;   // (a row may see nothing of its first tiles)
                if (seg_end < end) {      // the next segment's sequence and its query rows, now
                    int nb = b + 1;
                    while (P[nb + 1] <= seg_end) ++nb;
                    next = prefill_seq(p, nb);
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        if (r + 8 * half < next.qlen * p.group)
#pragma unroll
                            for (int x = 0; x < D * 2; x += 128)
                                asm volatile("prefetch.global.L1 [%0];" ::"l"(
                                    reinterpret_cast<const char *>(query_row(next, r + 8 * half)) + x));
                }
            }
            const int sg = i % nstages, k = i / nstages;
            ok = mbar_wait_warp(smem_addr(&bars[sg]), k & 1, p.status, &s_abort);
            if (!ok) break;
            unsigned char *kst = smem + sg * stage_bytes + warp * kHeadStride;   // this head
            const uint32_t kbase = smem_addr(kst);
            const int t0 = (g - P[b]) * kTT, valid = min(kTT, s.ctx - t0);
            if (valid > 0) {
                if (valid < kTT) {   // zero this head's V rows past the context (whole 128-byte rows)
                    for (int e = lane; e < kHalves * kTT * 8; e += 32) {
                        const int hh = e / (kTT * 8), row = (e % (kTT * 8)) / 8;
                        if (row >= valid)
                            *reinterpret_cast<uint4 *>(kst + v_off + hh * kHalfStride + row * 128 + (e % 8) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();   // (a later tile is copied over these rows)
                    __syncwarp();
                }
                warp_tile_attention<D, kTT, true, kF16>(st, qa, kbase, kbase + v_off, kHalfStride, tok_off, sees0 - t0,
                                                        sees1 - t0, sl2, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&bars[kMaxStages + sg]));
        }
        if (open && ok) close();
    }

    grid_dependents_launch();
    // Drain: wait (bounded) for the last phase of every stage this CTA armed.
    __syncthreads();
    if (threadIdx.x == 0) {
        const int issued = s_issued;
        for (int s = 0; s < nstages && s < issued; ++s) {
            const int k_last = (issued - 1 - s) / nstages;
            if (!mbar_wait(smem_addr(&bars[s]), k_last & 1)) record_status(p.status, kStatusTimeout);
        }
    }
}

// Join the pieces of each sequence cut between CTAs: a warp per (sequence, KV
// head, row), D / 32 dims a lane, pieces four at a time with every load of a
// group ahead of its use.
template <int D>
__global__ void __launch_bounds__(128)
prefill_rows_merge_kernel(const __grid_constant__ PrefillParams p, int ctas) {
    constexpr int E = D / 32;
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    const int w = blockIdx.y * 4 + (threadIdx.x >> 5), kvh = w >> 4, r = w & 15;
    const PrefillSeq s = prefill_seq(p, b);   // (written before the grid that this one waits for began)
    grid_dependency_wait();
    grid_dependents_launch();
    const int *P = p.tail_info;
    const int pb = P[b], pe = P[b + 1], W = P[p.num_seqs];
    if (pe == pb || kvh >= p.num_kv_heads || r >= s.qlen * p.group) return;
    const int C = min(ctas, W), c0 = rows_owner(pb, W, C), c1 = rows_owner(pe - 1, W, C);
    if (c0 == c1) return;   // held whole: written by its CTA
    float M = kLowestScore, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int base = c0; base <= c1; base += 4) {
        float m[4], l[4], o[4][E];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = kLowestScore;
            l[j] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[j][e] = 0.f;
            const int c = base + j;
            if (c > c1) continue;
            const int64_t row = piece_row(p, 2 * c + (rows_begin(c, W, C) >= pb ? 0 : 1), kvh, r);
            m[j] = __ldcg(p.part_max + row);
            l[j] = __ldcg(p.part_sum + row);
#pragma unroll
            for (int e = 0; e < E; ++e) o[j][e] = __ldcg(p.part_out + row * D + lane * E + e);
        }
        const float Mn = fmaxf(fmaxf(M, fmaxf(m[0], m[1])), fmaxf(m[2], m[3])), a = fast_exp2(M - Mn);
        M = Mn;
        L *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= a;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float wj = base + j <= c1 ? fast_exp2(m[j] - M) : 0.f;
            L = fmaf(wj, l[j], L);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wj, o[j][e], acc[e]);
        }
    }
    const float inv = L > 0.f ? 1.f / L : L;
    const int t = r / p.group;
    const int64_t at = (static_cast<int64_t>(s.q0 + t) * p.num_heads + kvh * p.group + (r - t * p.group)) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) store_pair_as(p.out, p.out_type, at + e, acc[e] * inv, acc[e + 1] * inv);
}

template <int D, bool kF16>
cudaError_t launch_rows(const PrefillParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                        cudaStream_t stream) {
    auto kern = prefill_rows_kernel<D, kF16>;
    const size_t fixed = 1024 + kRingBytes + 2 * kMaxStages * sizeof(uint64_t);
    static unsigned long long done = 0;
    cudaError_t e = ensure_smem_limit(kern, fixed + (2 * kPrefillRowsMaxSeqs + 1) * sizeof(int), done);
    if (e != cudaSuccess) return e;
    const dim3 grid(ctas, p.num_kv_heads / p.heads_per_cta);
    e = launch_kernel(kern, grid, dim3(32 * (p.heads_per_cta + 1)), fixed + (2 * p.num_seqs + 1) * sizeof(int), stream, 1u,
                      tk, tv, p);
    if (e != cudaSuccess) return e;
    return launch_kernel(prefill_rows_merge_kernel<D>, dim3(p.num_seqs, p.num_kv_heads * 4), dim3(128), 0, stream, 1u, p,
                         ctas);
}

}  // namespace

int prefill_rows_max() { return 16; }

cudaError_t launch_prefill_rows(const PrefillParams &p, bool f16, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                                cudaStream_t stream) {
    if (p.num_seqs > kPrefillRowsMaxSeqs || p.num_kv_heads > kPrefillRowsMaxKvHeads || p.heads_per_cta < 1 ||
        p.heads_per_cta > kMaxHeads)
        return cudaErrorInvalidValue;
    if (p.head_dim == 128)
        return f16 ? launch_rows<128, true>(p, tk, tv, ctas, stream) : launch_rows<128, false>(p, tk, tv, ctas, stream);
    return f16 ? launch_rows<64, true>(p, tk, tv, ctas, stream) : launch_rows<64, false>(p, tk, tv, ctas, stream);
}

}  // namespace pa
