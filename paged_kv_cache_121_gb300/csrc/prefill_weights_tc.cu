// The weights that several query tokens a sequence gave each cached token, on the
// fifth-generation tensor cores (tcgen05 + tensor memory): 16-bit caches, any block size.
//
// Mathematics: prefill_weights_simt.cu. Two passes, one skeleton: scores of 128 x 128
// (M = rows that are held, N = rows that are streamed, K = head_dim) land in tensor
// memory with a held row a lane, so that what is reduced over lies along a thread's own
// columns:
//  * statistics: query rows held, keys streamed; a thread keeps its row's running
//    maximum and sum;
//  * sums: keys held, query rows streamed; a thread adds up the rows' weights of its key.
//    Where a KV head has 128 query rows or less, they are the held side (and N) again: a
//    tile of keys is then done with its one product.
//
// Bound: the products and the exponentials, 512 cycles a tile each (two passes: twice
// the products and exponentials of one attention's scores), and in the sums as many for the
// rows' numbers, read from shared memory (sum_weights); for windows of few queries,
// reading K twice. So neither waits for the other. Persistent CTAs, one an SM, of
//  * warps 0-7 and 8-15: two groups, each with a tile of scores in work and one behind
//    it (4 x 128 columns of tensor memory), two warps a lane quarter, so that a scheduler
//    has four warps to hide an exponential's latency with;
//  * warp 16: issues the products;
//  * warp 17: draws the units, lays them out in a ring of shared memory for all others, and
//    fetches the tiles by TMA, in the 128-byte swizzled K-major operand's layout: blocks of
//    keys, whole tiles of query rows. That takes blocks of a power of two of 8 tokens or
//    more and 128 to be whole query tokens; else warps 17-20 fetch 32 rows of each tile,
//    gathered one by one, by 16-byte asynchronous copies (row r's chunk c at c ^ (r & 7)),
//    with up to two tiles of a warp on their way, each made visible to the tensor cores
//    (fence.proxy.async) before it is reported. The copies wait in the same queue as the
//    exponentials: a tile takes a warp 800 to 1,200 cycles. (TMA gathers of four rows
//    took 80 cycles each, 5,200 a tile.)
// A unit holds two tiles, one a group, so that a streamed tile feeds 256 held rows;
// where a KV head has 128 query rows or less, a unit holds those, and the groups take
// every other key tile (windows of 32 queries in 16 prompts: the sums 54 us with the
// keys held, two key tiles a unit for one of rows, and 42 so). Long units first; those of the sums, whose
// lengths differ most, are drawn from a counter, those of the statistics (cut into
// pieces of the context) go round the CTAs back and forth.
//
// Measured (GB300, 32 / 8 heads of 128). Windows of 32 queries, 16 prompts of 4,100
// tokens, bf16, blocks of 16: 80.3 us = statistics 40, between 5, sums 43 (each alone, under
// the profiler; bytes 45 and 42 %, tensor pipe 23 and 22 %, exponentials 25 and 22 %, issue
// slots 34 and 44 % of their rates: a tile comes in about 2,100 cycles, and its 16 boxes of
// 2 KB have a share in that, since with blocks of 128 a pass takes a quarter less; an L2 policy
// of evict-first or one more tile in flight change nothing). 8 chunks of 200 .. 1,500 tokens
// behind up to 2,500, fp16, blocks of 32: 174 us = 82 + 7 + 99 (tensor pipe 43 and 34 %,
// exponentials 46 and 35 %, issue slots 60 and 52 %; in a loop of calls 78, 5 and 95).
// Gathered by four copy warps (blocks of 24) the same two take 93 and 217 us. Of a first
// version, by one copy warp, with a warp a lane quarter and units as they are numbered, 171
// and 441.
//
// Every wait is bounded; on expiry the kernel records a timeout, waits (bounded) for its
// products and copies, frees its tensor memory and returns.
#include <algorithm>
#include <climits>

#include "async_copy.cuh"
#include "internal.h"
#include "packed_math.cuh"
#include "tcgen05.cuh"
#include "tile_ring.h"
#include "weights_common.cuh"

namespace pa {

namespace {

constexpr int kSide = 128;               // rows of a tile, either side
constexpr int kGroupWarps = 8;           // two for each 32 lanes of tensor memory: columns 0 .. 63 and 64 .. 127
constexpr int kMmaWarp = 2 * kGroupWarps;
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr int kCopyWarps = 4;            // that gather rows: 32 of every tile each
constexpr int kTileSpace = 192 * 1024;   // shared memory for tiles
constexpr int kMaxSlots = 12;
constexpr int kUnits = 4;                // units laid out ahead
constexpr int kLongUnit = 4;             // streamed tiles of a unit that is not fetched ahead
constexpr uint32_t kTmemCols = 512;

template <int D>
struct TcTile {
    static constexpr int kBytes = kSide * D * 2;
    static constexpr int kHalf = kSide * 128;          // one 64-dim half
    static constexpr int kSlots = kTileSpace / kBytes;
    static constexpr int kChunks = D / 8;              // 16-byte chunks of a row
    static_assert(kSlots <= kMaxSlots, "barriers for every slot");
};

// A unit of work.
struct Unit {
    int b, head, tile;   // the first of the held tiles (b negative: no more units)
    int held;            // tiles held: 1 or 2
    int piece;
    int lo, hi;          // streamed tiles
    int from[2], to[2];  // those that each group scores: from .. to - 1
    int rows;            // query rows of the KV head
    WeightSeq s;
};

struct Shared {
    uint64_t unit_full[kUnits], unit_empty[kUnits];
    uint64_t held_full[2][2], held_empty[2][2];   // [tile][buffer]
    uint64_t str_full[kMaxSlots], str_empty[kMaxSlots];
    uint64_t s_full[2][2], s_free[2][2];          // [group][buffer of scores]
    uint64_t part_full[2], part_free[2];          // [group]
    uint64_t done;
    uint32_t tmem;
    int abort_flag;
    Unit unit[kUnits];
    __align__(16) float minus[2 * kGroupWarps][kSide / 2], inverse[2 * kGroupWarps][kSide / 2];   // [warp]: of its columns' rows
    float part[2][kSide];                         // [group]: the sums over the second half of the columns
};

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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <bool kSums>
__host__ __device__ __forceinline__ int64_t unit_count(const PrefillWeightsParams &p) {
    const int64_t heads = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads;
    if (kSums && p.pair) return (static_cast<int64_t>(p.max_ctx) + 2 * kSide - 1) / (2 * kSide) * p.row_pieces * heads;
    const int64_t side = p.pair ? 2 * kSide : kSide;
    return (static_cast<int64_t>(p.max_count) * p.group + side - 1) / side * p.pieces * heads;
}

// The row tiles of a unit of keys, numbered (pair of key tiles x piece of the rows) x sequence: those that each
// group scores. False where there is nothing in it.
__device__ __forceinline__ bool lay_out_sums(const PrefillWeightsParams &p, int n, Unit &u) {
    const int order = n / p.num_seqs, pair = order / p.row_pieces;
    u.b = n - order * p.num_seqs;
    u.piece = order - pair * p.row_pieces;
    u.s = weight_seq(p, u.b);
    u.rows = u.s.count * p.group;
    const int row_tiles = (u.rows + kSide - 1) / kSide, key_tiles = (u.s.ctx + kSide - 1) / kSide;
    u.tile = pair * 2;
    u.lo = u.hi = 0;
    if (u.tile >= key_tiles) return false;
    u.held = min(2, key_tiles - u.tile);
    auto first = [&](int tile) {   // the first row tile that sees the key tile
        const int64_t token = static_cast<int64_t>(tile) * kSide - u.s.past;
        return token <= 0 ? 0 : token >= u.s.count ? row_tiles : static_cast<int>(token) * p.group / kSide;
    };
    const int from0 = first(u.tile), from1 = u.held > 1 ? first(u.tile + 1) : row_tiles;
    const int lo = min(from0, from1), per = (row_tiles - lo + p.row_pieces - 1) / p.row_pieces;
    u.lo = min(row_tiles, lo + u.piece * per);
    u.hi = min(row_tiles, u.lo + per);
    u.from[0] = max(from0, u.lo);
    u.from[1] = max(from1, u.lo);
    u.to[0] = u.to[1] = u.hi;
    return true;
}

// Unit number `at`, longest first; false where there is nothing in it. (Units, rows and keys fit 30 bits.)
template <bool kSums>
__device__ __forceinline__ bool lay_out(const PrefillWeightsParams &p, unsigned at, Unit &u) {
    if (kSums && p.pair) {
        const int n = static_cast<int>(at / static_cast<unsigned>(p.num_kv_heads));
        u.head = static_cast<int>(at) - n * p.num_kv_heads;
        return lay_out_sums(p, p.order ? p.order[n] : n, u);
    }
    const unsigned heads = p.num_seqs * p.num_kv_heads, order = at / heads, bh = at - order * heads;
    u.b = static_cast<int>(bh / static_cast<unsigned>(p.num_kv_heads));
    u.head = static_cast<int>(bh) - u.b * p.num_kv_heads;
    u.s = weight_seq(p, u.b);
    u.rows = u.s.count * p.group;
    const int row_tiles = (u.rows + kSide - 1) / kSide;
    // the last rows see most keys
    const int per_unit = p.pair ? 2 : 1;
    const int all = (p.max_count * p.group + per_unit * kSide - 1) / (per_unit * kSide);
    const int row_unit = static_cast<int>(order) / p.pieces;
    u.piece = static_cast<int>(order) - row_unit * p.pieces;
    u.tile = (all - 1 - row_unit) * per_unit;
    if (u.tile >= row_tiles) return false;
    u.held = min(per_unit, row_tiles - u.tile);
    auto end = [&](int tile) {     // one past the last key tile that the row tile sees
        const int row = min(u.rows, (tile + 1) * kSide) - 1;
        return ((kSums ? u.s.ctx : u.s.sees(row / p.group)) + kSide - 1) / kSide;   // (every key has a sum)
    };
    const int end0 = end(u.tile), end1 = u.held > 1 ? end(u.tile + 1) : 0;
    const int most = max(end0, end1), per = (most + p.pieces - 1) / p.pieces;
    u.lo = min(most, u.piece * per);
    u.hi = min(most, u.lo + per);
    u.from[0] = u.from[1] = u.lo;
    u.to[0] = p.pair ? min(u.hi, end0) : u.hi;
    u.to[1] = p.pair ? min(u.hi, end1) : u.hi;
    return true;
}

// mbar_try_wait, suspended until the phase completes or some 20 us are over: 20 warps that poll would take the issue
// slots of those that compute.
__device__ __forceinline__ bool mbar_doze(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_one(const PrefillWeightsParams &p, Shared *sh, uint64_t *bar, int parity) {
    if (mbar_doze(smem_addr(bar), parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!*reinterpret_cast<volatile int *>(&sh->abort_flag)) {
        if (mbar_doze(smem_addr(bar), parity)) return true;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            record_status(p.status, kStatusTimeout);
            *reinterpret_cast<volatile int *>(&sh->abort_flag) = 1;
        }
    }
    return false;
}
// A whole warp's wait: the answer is the same in all its lanes.
__device__ __forceinline__ bool wait_warp(const PrefillWeightsParams &p, Shared *sh, uint64_t *bar, int parity) {
    if (__all_sync(0xffffffffu, mbar_doze(smem_addr(bar), parity))) return true;
    return __all_sync(0xffffffffu, wait_one(p, sh, bar, parity));
}

// Sum of a key's weights from 32 columns' rows; kMasked: only over columns see .. end - 1 (the product of a row that is
// left out may be no number). kFolded: `minus` holds minus the rows' folded_stats, else minus their best scores.
// What the warp reads of its rows is read by every lane, 16 bytes in 4 cycles of the shared memory: the one number takes
// as long as the tile's exponentials, two took the keys-held pass of the ragged chunks from 92 us to 112.
template <bool kMasked, bool kFolded>
__device__ __forceinline__ float sum_weights(const float (&s)[32], const float *minus, const float *inverse, uint64_t scale2,
                                             int see, int end) {
    uint64_t acc[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(minus + c);
        const uint64_t s0 = pair(s[c], s[c + 1]), s1 = pair(s[c + 2], s[c + 3]), m0 = pair(m.x, m.y), m1 = pair(m.z, m.w);
        float e[4];
        unpair(kFolded ? fma2(s0, scale2, m0) : mul2(add2(s0, m0), scale2), e[0], e[1]);
        unpair(kFolded ? fma2(s1, scale2, m1) : mul2(add2(s1, m1), scale2), e[2], e[3]);
#pragma unroll
        for (int n = 0; n < 4; ++n) e[n] = fast_exp2(e[n]);
        if (!kFolded) {
            const float4 inv = *reinterpret_cast<const float4 *>(inverse + c);
            e[0] *= inv.x;
            e[1] *= inv.y;
            e[2] *= inv.z;
            e[3] *= inv.w;
        }
        if (kMasked) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (c + n < see || c + n >= end) e[n] = 0.f;
        }
        acc[0] = add2(acc[0], pair(e[0], e[1]));
        acc[1] = add2(acc[1], pair(e[2], e[3]));
    }
    float a, b;
    unpair(add2(acc[0], acc[1]), a, b);
    return a + b;
}

// A row's maximum (raw scores, times the scale's sign) and sum of 2^((s - best) * scale) go on with 32 keys.
template <bool kNegative>
__device__ __forceinline__ void add_stats(const float (&s)[32], uint64_t scale2, float scale, float &top, float &sum) {
    float best[4] = {top, top, top, top};
#pragma unroll
    for (int c = 0; c < 32; c += 8)
#pragma unroll
        for (int n = 0; n < 4; ++n)
            best[n] = kNegative ? max3(best[n], -s[c + 2 * n], -s[c + 2 * n + 1]) : max3(best[n], s[c + 2 * n], s[c + 2 * n + 1]);
    const float up = max3(fmaxf(best[0], best[1]), best[2], best[3]);
    const float ref = up == -INFINITY ? 0.f : up;   // (nothing seen yet: 2^-inf = 0)
    sum *= fast_exp2((top - ref) * fabsf(scale));
    top = up;
    const uint64_t minus = kNegative ? pair(ref, ref) : pair(-ref, -ref);
    uint64_t acc[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        float a, b;
        unpair(mul2(add2(pair(s[2 * c], s[2 * c + 1]), minus), scale2), a, b);
        acc[c & 1] = add2(acc[c & 1], pair(fast_exp2(a), fast_exp2(b)));
    }
    float a, b;
    unpair(add2(acc[0], acc[1]), a, b);
    sum += a + b;
}

template <bool kTma>
constexpr int kThreads = 32 * (kLoadWarp + (kTma ? 1 : kCopyWarps));

enum Pass { kStats, kSumsKeysHeld, kSumsRowsHeld };   // (the last: one row tile a KV head, as the statistics take it)
template <int D, bool kF16, bool kTma, int kPass>
__global__ void __launch_bounds__(kThreads<kTma>, 1)
prefill_weights_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ PrefillWeightsParams p, const int held_buffers) {
    using T = TcTile<D>;
    constexpr int kLoadWarps = kTma ? 1 : kCopyWarps;
    constexpr bool kSums = kPass != kStats;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *tiles = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Shared *sh = reinterpret_cast<Shared *>(tiles + kTileSpace);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool split = kSums ? kPass == kSumsRowsHeld : !p.pair;   // the groups take every other streamed tile of one held tile
    constexpr bool held_keys = kPass == kSumsKeysHeld;             // (the other operand is streamed)
    const int held_slots = (split ? 1 : 2) * held_buffers;
    const int str_slots = T::kSlots - held_slots;        // streamed tiles, behind the held ones

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2; ++j) {
                mbar_init(smem_addr(&sh->held_full[i][j]), kLoadWarps);
                mbar_init(smem_addr(&sh->held_empty[i][j]), 1);
                mbar_init(smem_addr(&sh->s_full[i][j]), 1);
                mbar_init(smem_addr(&sh->s_free[i][j]), kGroupWarps);
            }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh->part_full[i]), kGroupWarps / 2);
            mbar_init(smem_addr(&sh->part_free[i]), kGroupWarps / 2);
        }
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(smem_addr(&sh->unit_full[i]), 1);
            mbar_init(smem_addr(&sh->unit_empty[i]), 2 * kGroupWarps + 1 + kLoadWarps - 1);   // (all but the one that lays them out)
        }
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(smem_addr(&sh->str_full[i]), kLoadWarps);
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

    // unit k of this CTA, for a warp that has read what it needs of it
    auto unit_ready = [&](int k) { return wait_warp(p, sh, &sh->unit_full[k % kUnits], (k / kUnits) & 1); };
    auto unit_read = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh->unit_empty[k % kUnits]));
    };

    if (warp >= kLoadWarp) {
        // ---------------------------- units and tiles ----------------------------
        const int mine = warp - kLoadWarp;
        const uint32_t base = smem_addr(tiles) + mine * 32 * 128;   // (copies) this warp's rows of the first slot
        const uint64_t policy = l2_policy_evict_last();             // (both operands are read by many)
        uint64_t *pending = nullptr;   // the barrier of the tile that is on its way
        auto report = [&]() {          // its rows have arrived
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(pending));
            pending = nullptr;
        };
        // What others wait for is reported before this warp waits for them.
        auto wait_for = [&](uint64_t *bar, int parity) {
            if (pending && !__all_sync(0xffffffffu, mbar_test(smem_addr(bar), parity))) {
                copy_wait<0>();
                report();
            }
            return wait_warp(p, sh, bar, parity);
        };
        // Where the lane's part of a tile comes from. TMA: its box of keys (block, first token in it), or none; else its
        // row (none: zeros, as for a block outside the pool).
        struct Place {
            const uint16_t *row;
            int blk, at;
            bool live;
        };
        const int box = min(p.block_size, kSide);   // tokens of one box of keys
        auto locate = [&](const Unit &u, bool keys, int tile) {
            Place w{nullptr, 0, 0, false};
            if (kTma) {
                if (!keys) {
                    w.live = lane < D / 64;
                    w.at = u.s.q0 + tile * (kSide / p.group);
                } else {
                    const int t = tile * kSide + lane / (D / 64) * box, j = t / p.block_size;
                    w.live = t < min(u.s.ctx, (tile + 1) * kSide);
                    w.at = t - j * p.block_size;
                    if (w.live) w.blk = p.block_tables[static_cast<int64_t>(u.b) * p.max_blocks + j];
                }
                return w;
            }
            const int r = tile * kSide + mine * 32 + lane;
            if (keys && r < u.s.ctx) {
                const int j = r / p.block_size, blk = p.block_tables[static_cast<int64_t>(u.b) * p.max_blocks + j];
                if (static_cast<unsigned>(blk) < static_cast<unsigned>(p.num_blocks))
                    w.row = static_cast<const uint16_t *>(p.k_cache) +
                            ((static_cast<int64_t>(blk) * p.block_size + (r - j * p.block_size)) * p.num_kv_heads + u.head) * D;
            } else if (!keys && r < u.rows) {
                const int token = r / p.group;
                w.row = static_cast<const uint16_t *>(p.query) +
                        ((static_cast<int64_t>(u.s.q0) + token) * p.num_heads + u.head * p.group + r - token * p.group) * D;
            }
            return w;
        };
        // Fetch a tile once `empty` has completed the phase of this parity (negative: the slot is free).
        auto fetch = [&](const Unit &u, bool keys, const Place &w, int slot, uint64_t *full, uint64_t *empty, int parity) {
            if (parity >= 0 && !wait_for(empty, parity)) return false;
            if (kTma) {   // (boxes of keys past the context are left out: what the slot holds there is not looked at)
                const int half = lane % (D / 64), bytes = (keys ? box : kSide) * 128;
                const unsigned boxes = __popc(__ballot_sync(0xffffffffu, w.live));
                const uint32_t to = smem_addr(tiles) + slot * T::kBytes + half * T::kHalf, bar = smem_addr(full);
                if (lane == 0) mbar_arrive_expect_tx(bar, boxes * bytes);
                __syncwarp();
                if (w.live) {
                    if (keys) tma_load_5d(to + lane / (D / 64) * bytes, &map_k, 0, w.at, half, u.head, w.blk, bar, policy);
                    else tma_load_5d(to, &map_q, 0, half, 0, u.head, w.at, bar, policy);
                }
                return true;
            }
            const uint16_t *row = w.row;
            // A lane copies chunk c of every kStep-th row. Several rows' places are read at a time: a copy is ordered
            // behind the reads before it.
            constexpr int kStep = 32 / T::kChunks;
            const int r0 = lane / T::kChunks, c = lane % T::kChunks;
            const uint32_t to = base + slot * T::kBytes + (c >> 3) * T::kHalf + r0 * 128;
            const bool all = __all_sync(0xffffffffu, row != nullptr);
#pragma unroll
            for (int i0 = 0; i0 < T::kChunks; i0 += 8) {
                const uint16_t *src[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    src[i] = reinterpret_cast<const uint16_t *>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r0 + (i0 + i) * kStep));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t dst = to + (i0 + i) * kStep * 128 + (((c & 7) ^ ((r0 + (i0 + i) * kStep) & 7)) << 4);
                    if (all) copy16(dst, src[i] + c * 8);
                    else copy16_or_zeros(dst, src[i] ? src[i] + c * 8 : static_cast<const uint16_t *>(p.query), src[i] != nullptr);
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
        const unsigned units = static_cast<unsigned>(unit_count<kSums>(p));
        unsigned turn = 0, at = blockIdx.x;
        TileRing held_ring[2] = {TileRing(held_buffers), TileRing(held_buffers)}, str_ring(str_slots);
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (mine == 0) {
                // Long units of the sums are drawn, once the tiles of the one before are on their way: drawn earlier they
                // would wait here while other CTAs have none. Others go round the CTAs back and forth (a draw would
                // take as long as a short unit).
                const bool draws = held_keys && held_buffers == 1;
                bool found = false;
                while (!found && (at < units || (!draws && turn * gridDim.x < units))) {
                    if (at < units) found = lay_out<kSums>(p, at, u);
                    if (draws) {
                        if (lane == 0) at = gridDim.x + atomicAdd(p.counter, 1);
                        at = __shfl_sync(0xffffffffu, at, 0);
                    } else {
                        ++turn;
                        at = turn * gridDim.x + ((turn & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                    }
                }
                if (!found) u.b = -1;
                if (k >= kUnits && !wait_for(&sh->unit_empty[k % kUnits], (k / kUnits - 1) & 1)) break;
                if (lane == 0) {
                    sh->unit[k % kUnits] = u;
                    mbar_arrive(smem_addr(&sh->unit_full[k % kUnits]));
                }
            } else {
                if (!wait_for(&sh->unit_full[k % kUnits], (k / kUnits) & 1)) break;
                u = sh->unit[k % kUnits];
                unit_read(k);
            }
            if (u.b < 0) break;
            if (u.lo >= u.hi) continue;
            // (a tile's rows are looked up while the one before is sent for)
            const Place held[2] = {locate(u, held_keys, u.tile), locate(u, held_keys, u.held > 1 ? u.tile + 1 : u.tile)};
            Place next = locate(u, !held_keys, u.lo);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i >= u.held || !ok) break;
                const int buf = held_ring[i].slot();
                ok = fetch(u, held_keys, held[i], i * held_buffers + buf, &sh->held_full[i][buf], &sh->held_empty[i][buf],
                           held_ring[i].empty_parity());
                held_ring[i].count(ok);
            }
            for (int i = u.lo; i < u.hi && ok; ++i) {
                const Place here = next;
                if (i + 1 < u.hi) next = locate(u, !held_keys, i + 1);
                const int slot = str_ring.slot();
                ok = fetch(u, !held_keys, here, held_slots + slot, &sh->str_full[slot], &sh->str_empty[slot], str_ring.empty_parity());
                str_ring.count(ok);
            }
        }
        if (kTma) {   // nothing is on its way when the CTA ends: the last phase of every slot that was filled
            auto drain = [&](uint64_t *full, const TileRing &ring) {
                for (int i = ring.first_left(); i < ring.sent; ++i)
                    if (!mbar_wait(smem_addr(full + i % ring.slots), ring.full_parity(i))) record_status(p.status, kStatusTimeout);
            };
            if (lane == 0) {
                drain(sh->held_full[0], held_ring[0]);
                drain(sh->held_full[1], held_ring[1]);
                drain(sh->str_full, str_ring);
            }
            __syncwarp();
        } else {
            copy_wait<0>();
            if (pending) report();
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------ products ------------------------------
        constexpr uint32_t id = idesc_16bit_f32(kSide, kSide, false, false, kF16);
        const uint64_t first_tile = smem_desc_sw128(smem_addr(tiles), 16, 1024);
        auto tile_at = [&](int slot) { return first_tile + static_cast<uint32_t>(slot) * static_cast<uint32_t>(T::kBytes >> 4); };
        int holds[2] = {0, 0}, streamed = 0, count[2] = {0, 0};
        bool ok = true;
        for (int k = 0; ok && unit_ready(k); ++k) {
            const Unit *u = &sh->unit[k % kUnits];
            const int b = uniform(u->b), lo = uniform(u->lo), hi = uniform(u->hi), held = uniform(u->held);
            const int from[2] = {uniform(u->from[0]), uniform(u->from[1])}, to[2] = {uniform(u->to[0]), uniform(u->to[1])};
            unit_read(k);
            if (b < 0) break;
            if (lo >= hi) continue;
            int round[2], buf[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                round[i] = holds[i] / held_buffers;
                buf[i] = holds[i] - round[i] * held_buffers;
            }
            bool fine = true;
            if (elect_one()) {
                auto run = [&]() {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (i < held && !wait_one(p, sh, &sh->held_full[i][buf[i]], round[i] & 1)) return false;
                    int counted[2] = {count[0], count[1]}, slot = streamed % str_slots, phase = (streamed / str_slots) & 1;
                    for (int i = lo; i < hi; ++i) {
                        if (!wait_one(p, sh, &sh->str_full[slot], phase)) return false;
                        const uint64_t sd = tile_at(held_slots + slot);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            if (i < from[g] || i >= to[g] || (split && ((i - lo) & 1) != g)) continue;
                            const int c = counted[g]++;
                            if (c >= 2 && !wait_one(p, sh, &sh->s_free[g][c & 1], ((c >> 1) - 1) & 1)) return false;
                            tc_fence_after();
                            const uint64_t hd = tile_at(split ? buf[0] : g * held_buffers + buf[g]);
                            // what is reduced over lies along the columns: keys, in the sums rows
                            const uint64_t ad = kSums && split ? sd : hd, bd = kSums && split ? hd : sd;
                            const uint32_t to_col = tmem + static_cast<uint32_t>((2 * g + (c & 1)) * kSide);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t step = desc_step((kk / 4) * T::kHalf + (kk % 4) * 32);
                                tc_mma_16bit(to_col, ad + step, bd + step, id, kk > 0 ? 1u : 0u);
                            }
                            tc_commit(smem_addr(&sh->s_full[g][c & 1]));
                        }
                        tc_commit(smem_addr(&sh->str_empty[slot]));
                        if (++slot == str_slots) {
                            slot = 0;
                            phase ^= 1;
                        }
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
            for (int g = 0; g < 2; ++g)   // what the issuing lane counted
                count[g] += split ? (hi - lo + 1 - g) / 2 : max(0, min(to[g], hi) - max(from[g], lo));
        }
        if (elect_one()) {   // every product issued has run once `done` completes
            tc_commit(smem_addr(&sh->done));
            if (!mbar_wait(smem_addr(&sh->done), 0)) record_status(p.status, kStatusTimeout);
        }
        __syncwarp();
    } else {
        // ------------------------------ exponentials ------------------------------
        const int g = warp / kGroupWarps, h = (warp / 4) & 1, R = (warp & 3) * 32 + lane;   // group, half of the columns, lane
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
        int count = 0, joined = 0;   // tiles scored; sums put together
        bool ok = true, ahead = false;
        float next_off[2] = {0.f, 0.f};   // sums, keys held: folded_stats of two of this warp's columns in the next tile, once `ahead`
        bool folded = false;              // all of a tile's columns are
        float *const minus = sh->minus[warp], *const inverse = sh->inverse[warp];
        // A row's place among those of all KV heads.
        auto place = [&](const Unit *u, int r) {
            return u->s.stat0 * p.num_heads + u->head * p.group + r + static_cast<int64_t>(p.group_div.of(r)) * (p.num_heads - p.group);
        };
        auto columns = [&](const Unit *u, int i) {   // (loaded here, used a tile later)
            const int r = i * kSide + h * 64 + lane * 2, rows = u->rows;
#pragma unroll
            for (int n = 0; n < 2; ++n) next_off[n] = r + n < rows ? p.offsets[place(u, r + n)] : INFINITY;
            ahead = true;
        };
        auto lay_down_two_numbers = [&](const Unit *u, int i) {
            const int r = i * kSide + h * 64 + lane * 2, rows = u->rows;
            float2 row[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) row[n] = r + n < rows ? p.rows[place(u, r + n)] : make_float2(0.f, 0.f);
            *reinterpret_cast<float2 *>(minus + lane * 2) = make_float2(-row[0].x, -row[1].x);
            *reinterpret_cast<float2 *>(inverse + lane * 2) = make_float2(row[0].y, row[1].y);
        };
        auto lay_down_columns = [&](const Unit *u, int i) {
            folded = __all_sync(0xffffffffu, next_off[0] == next_off[0] && next_off[1] == next_off[1]);
            if (folded) *reinterpret_cast<float2 *>(minus + lane * 2) = make_float2(-next_off[0], -next_off[1]);
            else lay_down_two_numbers(u, i);
        };
        for (int k = 0; ok; ++k) {
            if (!unit_ready(k)) break;
            const Unit *u = &sh->unit[k % kUnits];   // (given back at the unit's end)
            if (u->b < 0) break;
            const int tile = split ? u->tile : u->tile + g;
            const int held_row = tile * kSide + R, rows = u->rows;
            float top = -INFINITY, sum = 0.f;   // statistics: maximum and sum; sums: the sum
            int row_sees = 0, first_row = 0;    // statistics: keys that the row sees; sums: the first row that sees the key
            int whole_from = 0, whole_to = 0;   // sums: row tiles whose rows all exist and see all of the key tile. (Rows past the
                                                //   last one are zeros, whose products with infinite keys are no numbers)
            if (!kSums && held_row < rows) row_sees = u->s.sees(held_row / p.group);
            auto key_tile = [&](int t) {
                const int64_t token = static_cast<int64_t>(t) * kSide + R - u->s.past;
                first_row = token <= 0 ? 0 : token >= u->s.count ? rows : static_cast<int>(token) * p.group;
                const int64_t all = static_cast<int64_t>(t + 1) * kSide - 1 - u->s.past;   // the first token that sees it all
                whole_to = (t + 1) * kSide <= u->s.ctx && all < u->s.count ? rows / kSide : 0;
                whole_from = all <= 0 || whole_to == 0 ? 0 : (static_cast<int>(all) * p.group + kSide - 1) / kSide;
            };
            auto weight_at = [&](int key) {
                return p.weights + (static_cast<int64_t>(u->b) * p.num_kv_heads + u->head) * p.weights_stride + key;
            };
            float old = 0.f;   // of the thread's key, on its way while the scores are
            auto look_up_old = [&](int key) {
                old = h == 0 && key < u->s.ctx && key < u->s.fresh && p.decay != 0.f ? *weight_at(key) : 0.f;
            };
            // The two halves of the columns.
            auto join = [&]() {
                if (h == 1) {
                    if (joined > 0 && !wait_warp(p, sh, &sh->part_free[g], (joined - 1) & 1)) return false;
                    sh->part[g][R] = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh->part_full[g]));
                } else {
                    if (!wait_warp(p, sh, &sh->part_full[g], joined & 1)) return false;
                    sum += sh->part[g][R];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh->part_free[g]));
                }
                ++joined;
                return true;
            };
            if (kSums && !split) key_tile(tile);
            if (kSums && split && u->lo < u->hi) {   // one tile of rows: their statistics serve the unit
                lay_down_two_numbers(u, u->tile);
                __syncwarp();
            }
            const int step = split ? 2 : 1, last = u->to[g];
            for (int i = u->from[g] + (split ? g : 0); i < last; i += step, ++count) {
                const int buf = count & 1;
                if (kSums && split) {
                    key_tile(i);
                    look_up_old(i * kSide + R);
                    sum = 0.f;
                } else if (kSums) {
                    if (!ahead) columns(u, i);
                    lay_down_columns(u, i);
                    ahead = false;
                    if (i + 1 < last) {
                        columns(u, i + 1);
                    } else {   // the next unit's first tile
                        if (!unit_ready(k + 1)) { ok = false; break; }
                        const Unit *next = &sh->unit[(k + 1) % kUnits];
                        if (next->b >= 0 && next->from[g] < next->to[g]) columns(next, next->from[g]);
                    }
                    __syncwarp();
                }
                if (!wait_warp(p, sh, &sh->s_full[g][buf], (count >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                const int row_tile = split ? tile : i;   // (of the sums)
                const bool whole = row_tile >= whole_from && row_tile < whole_to;
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    const int col = h * 64 + part * 32;
                    float s[32];
                    tmem_ld32(tmem + lane_off + static_cast<uint32_t>((2 * g + buf) * kSide + col), s);
                    if (part == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&sh->s_free[g][buf]));
                    }
                    const int c0 = (kSums ? row_tile : i) * kSide + col;   // the first column's row (statistics: key)
                    if (kSums) {
                        const float *const m = minus + part * 32, *const inv = inverse + part * 32;
                        if (held_keys && folded)
                            sum += whole ? sum_weights<false, true>(s, m, inv, scale2, 0, 32)
                                         : sum_weights<true, true>(s, m, inv, scale2, first_row - c0, rows - c0);
                        else if (!held_keys && whole)
                            sum += sum_weights<false, false>(s, m, inv, scale2, 0, 32);
                        else
                            sum += sum_weights<true, false>(s, m, inv, scale2, first_row - c0, rows - c0);
                    } else {
                        const bool negative = p.scale_log2 < 0.f;
                        if (__any_sync(0xffffffffu, c0 + 32 > row_sees)) {
                            const float masked = negative ? INFINITY : -INFINITY;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (c0 + c >= row_sees) s[c] = masked;
                        }
                        if (negative) add_stats<true>(s, scale2, p.scale_log2, top, sum);
                        else add_stats<false>(s, scale2, p.scale_log2, top, sum);
                    }
                }
                if (kSums && split) {
                    if (!join()) { ok = false; break; }
                    const int key = i * kSide + R;
                    if (h == 0 && key < u->s.ctx) *weight_at(key) = sum + p.decay * old;
                }
                if (kSums) __syncwarp();   // the columns' statistics have been read
            }
            if (!ok) break;
            if (kSums) {
                if (!split) {
                    look_up_old(p.row_pieces > 1 ? INT_MAX : held_row);
                    if (!join()) break;
                    if (h == 0 && g < u->held && held_row < u->s.ctx) {
                        if (p.row_pieces > 1)
                            p.parts[((static_cast<int64_t>(u->piece) * p.num_seqs + u->b) * p.num_kv_heads + u->head) * p.max_ctx + held_row] = sum;
                        else
                            *weight_at(held_row) = sum + p.decay * old;
                    }
                }
            } else if ((split || g < u->held) && held_row < rows) {
                const int token = held_row / p.group;
                leave_stats(p, 2 * (split ? 2 * u->piece + g : u->piece) + h, u->s.stat0 + token, u->head * p.group + held_row - token * p.group, top, sum);
            }
            unit_read(k);
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

// Between the passes: the rows' statistics put together; and, in the last CTA, the second pass's units in order of
// their length (to one of 256 lengths; which of equal ones is first does not show in the result), and its counter.
// Ragged chunks: the units as they are numbered leave the SMs idle for a third of the pass.
constexpr int kOrderThreads = 256;
__global__ void __launch_bounds__(kOrderThreads) weight_between_kernel(const __grid_constant__ PrefillWeightsParams p, int units) {
    __shared__ int start[256], scan[kOrderThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int t = threadIdx.x, lane = t & 31;
    if (blockIdx.x != gridDim.x - 1) {
        merge_stats(p, static_cast<int64_t>(blockIdx.x) * kOrderThreads + t);
        return;
    }
    if (t == 0) *p.counter = 0;
    if (!p.order) return;
    const int longest = max(1, static_cast<int>((static_cast<int64_t>(p.max_count) * p.group + kSide - 1) / kSide));
    auto bucket = [&](int n) {   // the longest in bucket 0, those with nothing in the last
        Unit u;
        const int len = lay_out_sums(p, n, u) ? u.hi - u.lo : -1;
        return len < 0 ? 255 : 254 - static_cast<int>(min(static_cast<int64_t>(254), static_cast<int64_t>(len) * 254 / longest));
    };
    start[t] = 0;
    __syncthreads();
    for (int n = t; n < units; n += kOrderThreads) atomicAdd(&start[bucket(n)], 1);
    __syncthreads();
    int sum = start[t];
    const int mine = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 31) scan[t >> 5] = sum;
    __syncthreads();
    int before = sum - mine;
    for (int w = 0; w < (t >> 5); ++w) before += scan[w];
    start[t] = before;
    __syncthreads();
    for (int n = t; n < units; n += kOrderThreads) p.order[atomicAdd(&start[bucket(n)], 1)] = n;
}

// The pieces of the rows put together: weights = decay * weights + their sums.
__global__ void __launch_bounds__(kOrderThreads) weight_parts_kernel(const __grid_constant__ PrefillWeightsParams p) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.y / p.num_kv_heads, t = blockIdx.x * kOrderThreads + threadIdx.x;
    const WeightSeq s = weight_seq(p, b);
    if (t >= s.ctx) return;
    const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads;
    float sum = 0.f;
    for (int i = 0; i < p.row_pieces; ++i) sum += p.parts[(i * rows + blockIdx.y) * p.max_ctx + t];
    float *w = p.weights + blockIdx.y * p.weights_stride + t;
    *w = sum + (t < s.fresh && p.decay != 0.f ? p.decay * *w : 0.f);
}

constexpr size_t kSmemBytes = 1024 + kTileSpace + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");

template <int D, bool kF16, bool kTma, int kPass>
cudaError_t launch_pass(const PrefillWeightsParams &p, const CUtensorMap &map_q, const CUtensorMap &map_k, int sms, cudaStream_t stream) {
    constexpr bool kSums = kPass != kStats;
    auto kern = prefill_weights_tc_kernel<D, kF16, kTma, kPass>;
    static unsigned long long done = 0;
    const cudaError_t e = ensure_smem_limit(kern, kSmemBytes, done);
    if (e != cudaSuccess) return e;
    // A unit that streams many tiles: more of them on their way. Short units: the next one's held tiles too.
    const int64_t streamed = kPass == kSumsKeysHeld ? (static_cast<int64_t>(p.max_count) * p.group + kSide - 1) / kSide
                                             : ((static_cast<int64_t>(p.max_ctx) + kSide - 1) / kSide + p.pieces - 1) / p.pieces;
    const int held_buffers = p.pair && streamed >= kLongUnit ? 1 : 2;
    return launch_kernel(kern, dim3(static_cast<unsigned>(std::min<int64_t>(unit_count<kSums>(p), sms))), dim3(kThreads<kTma>),
                         kSmemBytes, stream, 1u, map_q, map_k, p, held_buffers);
}

template <int D, bool kF16, bool kTma>
cudaError_t launch_both(const PrefillWeightsParams &p, const CUtensorMap &map_q, const CUtensorMap &map_k, int sms, cudaStream_t stream) {
    cudaError_t e = launch_pass<D, kF16, kTma, kStats>(p, map_q, map_k, sms, stream);
    if (e == cudaSuccess)
        e = launch_kernel(weight_between_kernel,
                          dim3(static_cast<unsigned>((p.stat_rows * p.num_heads + kOrderThreads - 1) / kOrderThreads + 1)),
                          dim3(kOrderThreads), 0, stream, 1u, p, static_cast<int>(unit_count<true>(p) / p.num_kv_heads));
    if (e == cudaSuccess)
        e = p.pair ? launch_pass<D, kF16, kTma, kSumsKeysHeld>(p, map_q, map_k, sms, stream)
                   : launch_pass<D, kF16, kTma, kSumsRowsHeld>(p, map_q, map_k, sms, stream);
    if (e != cudaSuccess || p.row_pieces == 1) return e;
    const dim3 grid(static_cast<unsigned>((p.max_ctx + kOrderThreads - 1) / kOrderThreads),
                    static_cast<unsigned>(p.num_seqs * p.num_kv_heads));
    return launch_kernel(weight_parts_kernel, grid, dim3(kOrderThreads), 0, stream, 1u, p);
}

}  // namespace

// Rows, keys and units have to fit 30 bits.
bool prefill_weights_tc_fits(int num_seqs, int num_kv_heads, int64_t rows, int max_ctx) {
    const int64_t most = int64_t(1) << 30, heads = static_cast<int64_t>(num_seqs) * num_kv_heads;
    return rows <= most - 2 * kSide && max_ctx <= most - 2 * kSide && heads < most &&
           ((rows + kSide - 1) / kSide + 1) * heads <= most / kMaxSplits && (max_ctx / (2 * kSide) + 1) * heads <= most;
}

// How the passes are cut. Statistics: rows of a unit, pieces of a context; a unit's time is its key tiles and some
// to begin and end with, and the pieces are those whose rounds over the SMs take least. Sums: pieces of the rows
// where the SMs would get fewer than kFewUnits units each.
constexpr int kFewUnits = 3;
constexpr int kMaxRowPieces = 8;
constexpr int64_t kMaxOrdered = 4096;   // units that one CTA puts in order
int64_t prefill_weights_tc_most_ordered() { return kMaxOrdered; }

void plan_prefill_weights_tc(int num_seqs, int num_kv_heads, int64_t rows, int max_ctx, int sms, int max_pieces,
                             int max_row_pieces, int *pair, int *pieces, int *row_pieces, int64_t *ordered) {
    *pair = rows > kSide;
    const int64_t side = *pair ? 2 * kSide : kSide, heads = static_cast<int64_t>(num_seqs) * num_kv_heads;
    const int64_t units = heads * ((rows + side - 1) / side);
    const int64_t tiles = (static_cast<int64_t>(max_ctx) + kSide - 1) / kSide;
    double best = 0;
    *pieces = 1;
    for (int n = 1; n <= kMaxSplits / 4 && n <= tiles && n <= max_pieces; ++n) {
        const double rounds = static_cast<double>((units * n + sms - 1) / sms);
        const double time = rounds * (static_cast<double>((tiles + n - 1) / n) * (*pair ? 2 : 1) + (*pair ? 3 : 1));
        if (n == 1 || time < best * 0.97) {
            best = time;
            *pieces = n;
        }
    }
    const int64_t key_units = (static_cast<int64_t>(max_ctx) + 2 * kSide - 1) / (2 * kSide) * heads;
    const int64_t row_tiles = (rows + kSide - 1) / kSide;
    *row_pieces = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>({(kFewUnits * sms + key_units - 1) / std::max<int64_t>(key_units, 1), row_tiles / 4, kMaxRowPieces,
                                  max_row_pieces})));
    if (heads > 65535) *row_pieces = 1;
    const int64_t n = key_units / num_kv_heads * *row_pieces;
    *ordered = row_tiles >= kLongUnit && n <= kMaxOrdered ? n : 0;   // (0: taken as they are numbered)
}

// Tokens of a box of keys and of a box of queries where tiles are fetched by TMA (else 0).
int prefill_weights_tc_key_box(int block_size) {
    return block_size >= 8 && (block_size & (block_size - 1)) == 0 ? std::min(block_size, kSide) : 0;
}
int prefill_weights_tc_query_box(int group) { return kSide % group == 0 ? kSide / group : 0; }

template <int D>
cudaError_t launch_dim(const PrefillWeightsParams &p, bool f16, bool tma, const CUtensorMap &map_q, const CUtensorMap &map_k, int sms,
                       cudaStream_t stream) {
    if (tma)
        return f16 ? launch_both<D, true, true>(p, map_q, map_k, sms, stream) : launch_both<D, false, true>(p, map_q, map_k, sms, stream);
    return f16 ? launch_both<D, true, false>(p, map_q, map_k, sms, stream) : launch_both<D, false, false>(p, map_q, map_k, sms, stream);
}

cudaError_t launch_prefill_weights_tc(const PrefillWeightsParams &p, bool f16, int head_dim, bool tma, const CUtensorMap &map_q,
                                      const CUtensorMap &map_k, int sms, cudaStream_t stream) {
    return head_dim == 128 ? launch_dim<128>(p, f16, tma, map_q, map_k, sms, stream)
                           : launch_dim<64>(p, f16, tma, map_q, map_k, sms, stream);
}

}  // namespace pa
