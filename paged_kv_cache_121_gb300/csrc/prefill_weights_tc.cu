// The weights that several query tokens a sequence gave each cached token, on the
// fifth-generation tensor cores (tcgen05 + tensor memory): 16-bit caches, any block size.
//
// Mathematics: prefill_weights_simt.cu. Two kernels, one skeleton: scores of 128 x 128
// (M = rows that are held, N = rows that are streamed, K = head_dim) land in tensor
// memory with a held row a lane, so that what is reduced over lies along a thread's own
// columns:
//  * statistics: query rows held, keys streamed; a thread keeps its row's running
//    maximum and sum of 2^(s - maximum);
//  * sums: keys held, query rows streamed; a thread adds up 2^(s - o_row) for its key.
//
// Bound: the exponentials, two a (row, key) pair at 16 a cycle and SM, four times the
// time of the products; for windows of few queries, reading K twice. So the tensor
// cores run ahead and the exponentials never wait: persistent CTAs, one an SM, of
//  * warps 0-3 and 4-7: two groups, each with a tile of scores in work and one behind
//    it (4 x 128 columns of tensor memory);
//  * warp 8: issues the products;
//  * warp 9: fetches the held tiles, warps 10 and 11 the streamed ones in turn, by 16-byte
//    asynchronous copies laid out as the 128-byte swizzled K-major operand (row r's chunk
//    c at c ^ (r & 7)): rows are gathered one by one, so blocks of any size and rows of
//    several query heads cost the same. A warp has up to two tiles on their way, and
//    makes a tile's copies visible to the tensor cores (fence.proxy.async) before it
//    reports it. Each slot is filled by one warp alone, so that the warp that waits for it
//    has seen every earlier phase of its barriers.
// A unit holds two tiles, one a group, so that a streamed tile feeds 256 held rows;
// where a KV head has 128 query rows or less, a unit of the statistics holds one, and
// the groups take every other key tile. Held tiles are double-buffered: the next unit's
// are fetched while this one's are in use. Units go round the CTAs back and forth,
// longest first.
// Every wait is bounded; on expiry the kernel records a timeout, waits (bounded) for its
// products, frees its tensor memory and returns.
#include <algorithm>

#include "internal.h"
#include "packed_math.cuh"
#include "tcgen05.cuh"
#include "weights_common.cuh"

namespace pa {

namespace {

constexpr int kSide = 128;               // rows of a tile, either side
constexpr int kGroupWarps = 4;
constexpr int kMmaWarp = 2 * kGroupWarps;
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr int kStreamWarps = 2;          // behind the one that fetches held tiles (12 warps: 168 registers a thread)
constexpr int kThreads = 32 * (kLoadWarp + 1 + kStreamWarps);
constexpr int kTileSpace = 192 * 1024;   // shared memory for tiles
constexpr int kMaxSlots = 12;
constexpr uint32_t kTmemCols = 512;

template <int D>
struct TcTile {
    static constexpr int kBytes = kSide * D * 2;
    static constexpr int kHalf = kSide * 128;          // one 64-dim half
    static constexpr int kSlots = kTileSpace / kBytes;
    static constexpr int kChunks = D / 8;              // 16-byte chunks of a row
    static_assert(kSlots <= kMaxSlots, "barriers for every slot");
    static_assert((kSlots - 2) % kStreamWarps == 0 && (kSlots - 4) % kStreamWarps == 0, "a streamed slot has one warp that fills it");
};

struct Shared {
    uint64_t held_full[2][2], held_empty[2][2];   // [tile][buffer]
    uint64_t str_full[kMaxSlots], str_empty[kMaxSlots];
    uint64_t s_full[2][2], s_free[2][2];       // [group][buffer of scores]
    uint64_t off_full[2][2];                   // [group][buffer of offsets]
    uint64_t done;
    uint32_t tmem;
    int abort_flag;
    __align__(16) float off[2][2][kSide];      // [group][buffer]: what to take from the scores of each streamed row
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
    const int bytes = live ? 16 : 0;   // (the rest is filled with zeros)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Whether the phase of this parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A unit of work, the same in every thread.
struct Unit {
    int k;             // its place in the CTA's list (negative: none)
    int b, head, tile; // the first of the held tiles
    int held;          // tiles held: 1 or 2
    int piece;
    int lo, hi;        // streamed tiles
    int from0, from1, to0, to1;   // those that each group scores: from .. to - 1
    WeightSeq s;
    __device__ __forceinline__ int from(int g) const { return g ? from1 : from0; }
    __device__ __forceinline__ int to(int g) const { return g ? to1 : to0; }
};

template <bool kSums>
__host__ __device__ __forceinline__ int64_t unit_count(const PrefillWeightsParams &p) {
    const int64_t heads = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads;
    if (kSums) return (static_cast<int64_t>(p.max_ctx) + 2 * kSide - 1) / (2 * kSide) * heads;
    const int64_t side = p.pair ? 2 * kSide : kSide;
    return (static_cast<int64_t>(p.max_count) * p.group + side - 1) / side * p.pieces * heads;
}

// The CTA's next unit with anything in it, from place k on. (Units, rows and keys fit 30 bits.)
template <bool kSums>
__device__ __forceinline__ Unit next_unit(const PrefillWeightsParams &p, int k) {
    const unsigned heads = p.num_seqs * p.num_kv_heads, units = static_cast<unsigned>(unit_count<kSums>(p));
    Unit u;
    for (;; ++k) {
        u.k = -1;
        if (k * gridDim.x >= units) return u;
        const unsigned at = k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        if (at >= units) continue;
        const unsigned order = at / heads, bh = at - order * heads;
        u.b = static_cast<int>(bh / static_cast<unsigned>(p.num_kv_heads));
        u.head = static_cast<int>(bh) - u.b * p.num_kv_heads;
        u.s = weight_seq(p, u.b);
        const int rows = u.s.count * p.group;
        const int row_tiles = (rows + kSide - 1) / kSide, key_tiles = (u.s.ctx + kSide - 1) / kSide;
        if (kSums) {   // the first keys are seen by most rows
            u.tile = static_cast<int>(order) * 2;
            if (u.tile >= key_tiles) continue;
            u.held = min(2, key_tiles - u.tile);
            u.piece = 0;
            auto first = [&](int tile) {   // the first row tile that sees the key tile
                const int64_t token = static_cast<int64_t>(tile) * kSide - u.s.past;
                return token <= 0 ? 0 : token >= u.s.count ? row_tiles : static_cast<int>(token) * p.group / kSide;
            };
            u.from0 = first(u.tile);
            u.from1 = u.held > 1 ? first(u.tile + 1) : row_tiles;
            u.hi = u.to0 = u.to1 = row_tiles;
            u.lo = min(u.from0, u.from1);
        } else {       // the last rows see most keys
            const int per_unit = p.pair ? 2 : 1;
            const int all = (p.max_count * p.group + per_unit * kSide - 1) / (per_unit * kSide);
            const int row_unit = static_cast<int>(order) / p.pieces;
            u.piece = static_cast<int>(order) - row_unit * p.pieces;
            u.tile = (all - 1 - row_unit) * per_unit;
            if (u.tile >= row_tiles) continue;
            u.held = min(per_unit, row_tiles - u.tile);
            auto end = [&](int tile) {     // one past the last key tile that the row tile sees
                const int row = min(rows, (tile + 1) * kSide) - 1;
                return (u.s.sees(row / p.group) + kSide - 1) / kSide;
            };
            const int end0 = end(u.tile), end1 = u.held > 1 ? end(u.tile + 1) : 0;
            const int most = max(end0, end1), per = (most + p.pieces - 1) / p.pieces;
            u.lo = min(most, u.piece * per);
            u.hi = min(most, u.lo + per);
            u.from0 = u.from1 = u.lo;
            u.to0 = p.pair ? min(u.hi, end0) : u.hi;
            u.to1 = p.pair ? min(u.hi, end1) : u.hi;
        }
        u.k = k;
        return u;
    }
}

__device__ __forceinline__ bool wait_one(const PrefillWeightsParams &p, Shared *sh, uint64_t *bar, int parity) {
    if (*reinterpret_cast<volatile int *>(&sh->abort_flag)) return false;
    if (mbar_wait(smem_addr(bar), parity)) return true;
    record_status(p.status, kStatusTimeout);
    *reinterpret_cast<volatile int *>(&sh->abort_flag) = 1;
    return false;
}
__device__ __forceinline__ bool wait_warp(const PrefillWeightsParams &p, Shared *sh, uint64_t *bar, int parity) {
    return mbar_wait_warp(smem_addr(bar), parity, p.status, &sh->abort_flag);
}

template <int D, bool kF16, bool kSums>
__global__ void __launch_bounds__(kThreads, 1)
prefill_weights_tc_kernel(const __grid_constant__ PrefillWeightsParams p) {
    using T = TcTile<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *tiles = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Shared *sh = reinterpret_cast<Shared *>(tiles + kTileSpace);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_unit = kSums || p.pair ? 2 : 1;
    const int str_slots = T::kSlots - 2 * per_unit;      // streamed tiles, behind two buffers of held ones

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            for (int j = 0; j < 2; ++j) {
                mbar_init(smem_addr(&sh->held_full[i][j]), 1);
                mbar_init(smem_addr(&sh->held_empty[i][j]), 1);
                mbar_init(smem_addr(&sh->s_full[i][j]), 1);
                mbar_init(smem_addr(&sh->s_free[i][j]), kGroupWarps);
                mbar_init(smem_addr(&sh->off_full[i][j]), kGroupWarps);
            }
        }
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(smem_addr(&sh->str_full[i]), 1);
            mbar_init(smem_addr(&sh->str_empty[i]), 1);
        }
        mbar_init(smem_addr(&sh->done), 1);
        sh->abort_flag = 0;
        mbar_fence_init();
    }
    grid_dependency_wait();
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&sh->tmem), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    // scores of group g, buffer n
    auto s_col = [&](int g, int n) { return tmem + static_cast<uint32_t>((2 * g + n) * kSide); };

    if (warp >= kLoadWarp) {
        // -------------------------------- loaders --------------------------------
        const bool holds = warp == kLoadWarp;
        const int mine = warp - kLoadWarp - 1;
        bool ok = true;
        uint64_t *pending = nullptr;   // the barrier of the tile that is on its way
        auto report = [&]() {          // the pending tile has arrived
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(pending));
            pending = nullptr;
        };
        // Fetch a tile into dst once `empty` has completed the phase of this parity (negative: it is free).
        auto fetch = [&](const Unit &u, bool keys, int tile, uint32_t dst, uint64_t *full, uint64_t *empty, int parity) {
            if (parity >= 0) {
                if (pending && !__all_sync(0xffffffffu, mbar_test(smem_addr(empty), parity))) {
                    copy_wait<0>();   // what the others wait for is reported before this warp waits for them
                    report();
                }
                if (!wait_warp(p, sh, empty, parity)) return false;
            }
            const int rows = u.s.count * p.group;
            const uint16_t *row[4];
            if (keys) {
                const int32_t *table = p.block_tables + static_cast<int64_t>(u.b) * p.max_blocks;
                int blk[4], at[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int t = tile * kSide + n * 32 + lane;
                    at[n] = t < u.s.ctx ? t % p.block_size : 0;
                    blk[n] = t < u.s.ctx ? table[t / p.block_size] : -1;
                }
#pragma unroll
                for (int n = 0; n < 4; ++n)   // (a block outside the pool reads as zeros)
                    row[n] = static_cast<unsigned>(blk[n]) < static_cast<unsigned>(p.num_blocks)
                                 ? static_cast<const uint16_t *>(p.k_cache) +
                                       ((static_cast<int64_t>(blk[n]) * p.block_size + at[n]) * p.num_kv_heads + u.head) * D
                                 : nullptr;
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int r = tile * kSide + n * 32 + lane, token = r / p.group;
                    row[n] = r < rows ? static_cast<const uint16_t *>(p.query) +
                                            ((static_cast<int64_t>(u.s.q0) + token) * p.num_heads + u.head * p.group + r - token * p.group) * D
                                      : nullptr;
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
#pragma unroll
                for (int i = 0; i < T::kChunks; ++i) {
                    const int at = i * 32 + lane, r = at / T::kChunks, c = at % T::kChunks;
                    const uint16_t *src = reinterpret_cast<const uint16_t *>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row[n]), r));
                    const int R = n * 32 + r;
                    copy16(dst + (c >> 3) * T::kHalf + R * 128 + (((c & 7) ^ (R & 7)) << 4),
                           src ? src + c * 8 : static_cast<const uint16_t *>(p.query), src != nullptr);
                }
            }
            copy_commit();
            if (pending) {
                copy_wait<1>();
                report();
            }
            pending = full;
            return true;
        };
        const uint32_t base = smem_addr(tiles);
        int held[2] = {0, 0}, streamed = 0;
        for (Unit u = next_unit<kSums>(p, 0); u.k >= 0 && ok; u = next_unit<kSums>(p, u.k + 1)) {
            if (u.lo >= u.hi) continue;
            if (holds) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (i >= u.held || !ok) break;
                    const int n = held[i]++, buf = n & 1;
                    ok = fetch(u, kSums, u.tile + i, base + (2 * i + buf) * T::kBytes, &sh->held_full[i][buf],
                               &sh->held_empty[i][buf], n >= 2 ? ((n >> 1) - 1) & 1 : -1);
                }
                continue;
            }
            for (int i = u.lo + ((mine ^ streamed) & 1); i < u.hi && ok; i += kStreamWarps) {
                const int n = streamed + i - u.lo, slot = n % str_slots, round = n / str_slots;
                ok = fetch(u, !kSums, i, base + (2 * per_unit + slot) * T::kBytes, &sh->str_full[slot], &sh->str_empty[slot],
                           round > 0 ? (round - 1) & 1 : -1);
            }
            streamed += u.hi - u.lo;
        }
        copy_wait<0>();
        if (pending) report();
    } else if (warp == kMmaWarp) {
        // ------------------------------ products ------------------------------
        constexpr uint32_t id = idesc_16bit_f32(kSide, kSide, false, false, kF16);
        const uint64_t first_tile = smem_desc_sw128(smem_addr(tiles), 16, 1024);
        int holds[2] = {0, 0}, streamed = 0, count[2] = {0, 0};
        bool ok = true;
        for (Unit u = next_unit<kSums>(p, 0); u.k >= 0 && ok; u = next_unit<kSums>(p, u.k + 1)) {
            const int lo = uniform(u.lo), hi = uniform(u.hi), held = uniform(u.held);
            if (lo >= hi) continue;
            const int buf[2] = {holds[0] & 1, holds[1] & 1};
            const int from[2] = {uniform(u.from0), uniform(u.from1)}, to[2] = {uniform(u.to0), uniform(u.to1)};
            int counted[2] = {count[0], count[1]};
            bool fine = true;
            if (elect_one()) {
                auto run = [&]() {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (i < held && !wait_one(p, sh, &sh->held_full[i][buf[i]], (holds[i] >> 1) & 1)) return false;
                    int n = streamed;
                    for (int i = lo; i < hi; ++i, ++n) {
                        const int slot = n % str_slots;
                        if (!wait_one(p, sh, &sh->str_full[slot], (n / str_slots) & 1)) return false;
                        const uint64_t sd = first_tile + static_cast<uint32_t>(2 * per_unit + slot) * static_cast<uint32_t>(T::kBytes >> 4);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            if (i < from[g] || i >= to[g] || !(kSums || p.pair || ((i - lo) & 1) == g)) continue;
                            const int c = counted[g]++;
                            if (c >= 2 && !wait_one(p, sh, &sh->s_free[g][c & 1], ((c >> 1) - 1) & 1)) return false;
                            tc_fence_after();
                            const int tile = per_unit == 2 ? 2 * g + buf[g] : buf[0];
                            const uint64_t hd = first_tile + static_cast<uint32_t>(tile) * static_cast<uint32_t>(T::kBytes >> 4);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t step = desc_step((kk / 4) * T::kHalf + (kk % 4) * 32);
                                tc_mma_16bit(s_col(g, c & 1), hd + step, sd + step, id, kk > 0 ? 1u : 0u);
                            }
                            tc_commit(smem_addr(&sh->s_full[g][c & 1]));
                        }
                        tc_commit(smem_addr(&sh->str_empty[slot]));
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (i < held) tc_commit(smem_addr(&sh->held_empty[i][buf[i]]));
                    return true;
                };
                fine = run();
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, fine);
            streamed += hi - lo;
            ++holds[0];
            holds[1] += held > 1;
#pragma unroll
            for (int g = 0; g < 2; ++g) {   // what the issuing lane counted
                const int n = max(0, min(to[g], hi) - max(from[g], lo));
                count[g] += kSums || p.pair ? n : (hi - lo + 1 - g) / 2;
            }
        }
        if (elect_one()) {   // every product issued has run once `done` completes
            tc_commit(smem_addr(&sh->done));
            if (!mbar_wait(smem_addr(&sh->done), 0)) record_status(p.status, kStatusTimeout);
        }
        __syncwarp();
    } else {
        // ------------------------------ exponentials ------------------------------
        const int g = warp / kGroupWarps, R = (warp & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
        int count = 0;   // tiles scored
        bool ok = true;
        float next_off = INFINITY;
        // this thread's column of streamed tile i (sums: a query row)
        auto column = [&](const Unit &u, int i) {
            const int r = i * kSide + R, token = r / p.group;
            const bool live = token < u.s.count;
            next_off = live ? row_offset(p, u.s.stat0 + token, u.head * p.group + r - token * p.group) : INFINITY;
        };
        Unit u = next_unit<kSums>(p, 0);
        if (kSums && u.k >= 0 && u.from(g) < u.to(g)) column(u, u.from(g));
        while (u.k >= 0 && ok) {
            const Unit next = next_unit<kSums>(p, u.k + 1);
            const int tile = kSums || p.pair ? u.tile + g : u.tile;
            const int held_row = tile * kSide + R;
            float top = -INFINITY, sum = 0.f;   // statistics: maximum and sum; sums: the sum
            int row_sees = 0, first_row = 0;    // statistics: keys that the row sees; sums: the first row that sees the key
            if (!kSums && held_row < u.s.count * p.group) row_sees = u.s.sees(held_row / p.group);
            if (kSums) {
                const int64_t token = static_cast<int64_t>(held_row) - u.s.past;
                first_row = token <= 0 ? 0 : token >= u.s.count ? u.s.count * p.group : static_cast<int>(token) * p.group;
            }
            const int step = kSums || p.pair ? 1 : 2, last = u.to(g);
            for (int i = u.from(g) + (step == 2 ? g : 0); i < last; i += step, ++count) {
                const int buf = count & 1;
                if (kSums) {
                    sh->off[g][buf][R] = next_off;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh->off_full[g][buf]));
                    if (i + 1 < last) column(u, i + 1);
                    else if (next.k >= 0 && next.from(g) < next.to(g)) column(next, next.from(g));
                    if (!wait_warp(p, sh, &sh->off_full[g][buf], (count >> 1) & 1)) { ok = false; break; }
                }
                if (!wait_warp(p, sh, &sh->s_full[g][buf], (count >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float s[64];
                    tmem_ld64(tmem + lane_off + static_cast<uint32_t>((2 * g + buf) * kSide + half * 64), s);
                    if (half == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&sh->s_free[g][buf]));
                    }
                    if (kSums) {
                        const float *off = &sh->off[g][buf][half * 64];
                        // the tile's first row sees least; rows past the last one are zeros, whose products
                        // with an infinite key are no numbers: they see nothing
                        const bool whole = (i + 1) * kSide <= u.s.count * p.group && (tile + 1) * kSide <= u.s.sees(i * kSide / p.group);
                        const int c0 = i * kSide + half * 64, see = first_row - c0, end = u.s.count * p.group - c0;
                        uint64_t acc[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < 64; c += 4) {
                            const float4 o = *reinterpret_cast<const float4 *>(off + c);
                            float e[4];
                            unpair(fma2(pair(s[c], s[c + 1]), scale2, pair(-o.x, -o.y)), e[0], e[1]);
                            unpair(fma2(pair(s[c + 2], s[c + 3]), scale2, pair(-o.z, -o.w)), e[2], e[3]);
#pragma unroll
                            for (int n = 0; n < 4; ++n) e[n] = fast_exp2(e[n]);
                            if (!whole) {
#pragma unroll
                                for (int n = 0; n < 4; ++n)
                                    if (c + n < see || c + n >= end) e[n] = 0.f;
                            }
                            acc[0] = add2(acc[0], pair(e[0], e[1]));
                            acc[1] = add2(acc[1], pair(e[2], e[3]));
                        }
                        float a, b;
                        unpair(add2(acc[0], acc[1]), a, b);
                        sum += a + b;
                    } else {
                        const int t0 = i * kSide + half * 64;
                        uint64_t x[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] = mul2(pair(s[2 * c], s[2 * c + 1]), scale2);
                        if (__any_sync(0xffffffffu, t0 + 64 > row_sees)) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                float a, b;
                                unpair(x[c], a, b);
                                x[c] = pair(t0 + 2 * c < row_sees ? a : -INFINITY, t0 + 2 * c + 1 < row_sees ? b : -INFINITY);
                            }
                        }
                        float best[4] = {top, top, top, top};
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            float a, b;
                            unpair(x[c], a, b);
                            best[c & 3] = fmaxf(best[c & 3], fmaxf(a, b));
                        }
                        const float up = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
                        const float ref = up == -INFINITY ? 0.f : up;   // (nothing seen yet: 2^-inf = 0)
                        sum *= fast_exp2(top - ref);
                        top = up;
                        const uint64_t minus = pair(-ref, -ref);
                        uint64_t acc[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            float a, b;
                            unpair(add2(x[c], minus), a, b);
                            acc[c & 1] = add2(acc[c & 1], pair(fast_exp2(a), fast_exp2(b)));
                        }
                        float a, b;
                        unpair(add2(acc[0], acc[1]), a, b);
                        sum += a + b;
                    }
                }
            }
            if (!ok) break;
            // (a unit that this group has nothing of did not look ahead)
            if (kSums && u.from(g) >= last && next.k >= 0 && next.from(g) < next.to(g)) column(next, next.from(g));
            if (kSums) {
                if (g < u.held && held_row < u.s.ctx) {
                    float *w = p.weights + (static_cast<int64_t>(u.b) * p.num_kv_heads + u.head) * p.weights_stride + held_row;
                    *w = sum + (held_row < u.s.fresh && p.decay != 0.f ? p.decay * *w : 0.f);
                }
            } else if ((!p.pair || g < u.held) && held_row < u.s.count * p.group) {
                const int token = held_row / p.group;
                const int slot = p.pair ? u.piece : 2 * u.piece + g;
                p.stats[(slot * p.stat_rows + u.s.stat0 + token) * p.num_heads + u.head * p.group + held_row - token * p.group] =
                    make_float2(top, sum);
            }
            u = next;
        }
    }
    tc_fence_before();
    __syncthreads();
    grid_dependents_launch();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

constexpr size_t kSmemBytes = 1024 + kTileSpace + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");

template <int D, bool kF16, bool kSums>
cudaError_t launch_one(const PrefillWeightsParams &p, int sms, cudaStream_t stream) {
    auto kern = prefill_weights_tc_kernel<D, kF16, kSums>;
    static unsigned long long done = 0;
    const cudaError_t e = ensure_smem_limit(kern, kSmemBytes, done);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(static_cast<unsigned>(std::min<int64_t>(unit_count<kSums>(p), sms))), dim3(kThreads), kSmemBytes, stream, 1u, p);
}

template <int D, bool kF16>
cudaError_t launch_both(const PrefillWeightsParams &p, int sms, cudaStream_t stream) {
    const cudaError_t e = launch_one<D, kF16, false>(p, sms, stream);
    return e != cudaSuccess ? e : launch_one<D, kF16, true>(p, sms, stream);
}

}  // namespace

// Rows, keys and units have to fit 30 bits.
bool prefill_weights_tc_fits(int num_seqs, int num_kv_heads, int64_t rows, int max_ctx) {
    const int64_t most = int64_t(1) << 30, heads = static_cast<int64_t>(num_seqs) * num_kv_heads;
    return rows <= most - 2 * kSide && max_ctx <= most - 2 * kSide && heads < most &&
           ((rows + kSide - 1) / kSide + 1) * heads <= most / kMaxSplits && (max_ctx / (2 * kSide) + 1) * heads <= most;
}

// How the statistics are cut: rows of a unit, pieces of a context. A unit's time is its key tiles, and
// half a tile to begin and end; the pieces are those whose rounds over the SMs take least.
void plan_prefill_weights_tc(int num_seqs, int num_kv_heads, int64_t rows, int max_ctx, int sms, int *pair, int *pieces) {
    *pair = rows > kSide;
    const int64_t side = *pair ? 2 * kSide : kSide;
    const int64_t units = static_cast<int64_t>(num_seqs) * num_kv_heads * ((rows + side - 1) / side);
    const int64_t tiles = (static_cast<int64_t>(max_ctx) + kSide - 1) / kSide;
    double best = 0;
    *pieces = 1;
    for (int n = 1; n <= kMaxSplits / 2 && n <= tiles; ++n) {
        const double rounds = static_cast<double>((units * n + sms - 1) / sms);
        const double time = rounds * (static_cast<double>((tiles + n - 1) / n) * (*pair ? 2 : 1) + 0.5);
        if (n == 1 || time < best * 0.97) {
            best = time;
            *pieces = n;
        }
    }
}

cudaError_t launch_prefill_weights_tc(const PrefillWeightsParams &p, bool f16, int head_dim, int sms, cudaStream_t stream) {
    if (head_dim == 128) return f16 ? launch_both<128, true>(p, sms, stream) : launch_both<128, false>(p, sms, stream);
    return f16 ? launch_both<64, true>(p, sms, stream) : launch_both<64, false>(p, sms, stream);
}

}  // namespace pa
