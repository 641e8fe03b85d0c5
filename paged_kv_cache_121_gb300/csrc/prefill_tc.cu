// Attention of several query tokens a sequence on the fifth-generation tensor
// cores (tcgen05 + tensor memory), sm_103a: 16-bit caches, paged in blocks of
// 8 to 256 tokens (powers of two) or contiguous.
//
// Mathematics: O = softmax(scale Q K^T + mask) V, the softmax held as a running
// maximum m and sum l of base-2 exponentials while 128-token K/V tiles stream
// past. m only moves when a score passes it by more than 2^8 (then O and l are
// rescaled): the result is the same, O is almost never touched. (Computing a
// tile's first weights with the maximum so far while its own is still being found
// was 6-12 % slower: both groups then want the exponential unit at once.)
//
// Rows. A row is (query token, query head); a KV head's rows are packed token
// by token, heads_per_tile heads each, into tiles of at most 128 rows, one
// tensor-memory lane each, so that a K/V tile is read once for all of them.
// A unit of work is one (row tiles, KV head):
//  * kTwoTiles: two row tiles share every K/V tile (many query tokens: bound by
//    the matrix products, 256 rows to a K/V byte);
//  * else one row tile whose K/V tiles the two softmax groups take in turn (few
//    query tokens: bound by the cache's bytes), joined in the epilogue.
// Either way two softmax groups of four warps alternate on the tensor cores:
// while one group turns its scores into weights, the other's products run.
//
// CTA (12 warps, one CTA per SM, persistent over units):
//  * warps 0-3, 4-7: softmax group 0, 1. One row a thread: scores from tensor
//    memory, weights back into the same columns as the 16-bit A operand of the
//    second product (no shared memory in between), then the epilogue.
//  * warp 8: issues the MMAs: per tile S = Q K^T (128 x 128 x D) and O += P V
//    (128 x D x 128). A group's next S overwrites its P: both run on the one
//    tensor pipe in issue order.
//  * warps 9, 10: K tiles, 64 tokens each; warp 11: the schedule, Q and V
//    tiles. TMA boxes, one per cache block (at most 64 tokens); K one box per
//    64-dim half, V too where blocks are long, else both halves in one. A thread
//    starts a box every ~50 ns, so blocks of 16 need three issuing warps.
//
// Bound: the tensor pipe, 79 % busy on long contexts (ncu; the rest is the hand-over
// between products and softmax, and the start and end of a unit). Measured on
// GB300, head_dim 128, causal, in a loop of calls on alternating inputs / as the
// best of a few short CUDA graphs: 2,048 tokens behind 30,720, 64 / 8 heads, 1,354 /
// 1,230 us (1,573 / 1,730 TFLOP/s, where cuBLAS sustains 1,697); four prompts of
// 4,100, 32 / 8 heads, 403 / 375 us (1,368 / 1,470); 64 chunks of 1 to 512 behind up
// to 3,584, 439 / 407 us (1,152 / 1,243). The two differ by the clock under the power
// limit. A tile takes about 2,500 cycles (its products 2,048), a change of unit 4,500
// to 5,500 (stamped before the epilogue's last step). At head_dim 64 neither the
// tensor pipe nor the exponential unit is above 47 %: a tile is paced by a group's
// chain of product, load, maximum, weights, product.
//
// Schedule: whole units, each CTA drawing the next as it goes (with a workspace and
// more than two waves of units; else CTA c takes c, c + C, ...): the CTAs then work
// on neighbouring units, which share their K and V, at any time. Where the host
// allows, the units of the last partial wave are cut where that pays: into pieces of
// units, one a CTA, or equal ranges of tiles over all CTAs; pieces of a unit go to the
// workspace for the merge kernel. (192 units of 64 tiles at head_dim 128: 196 us whole,
// 157 in pieces, 154 in ranges; 272 units of 12 tiles: 51 whole, 71 in ranges. All units
// cut into one contiguous range a CTA, measured: 64 ragged chunks 609 us against
// 450, four 4,100-token prompts 517 against 396: each CTA then streams a K and V of
// its own, and ranges of many short units take longer.)
//
// Tokens past a context's end: K's are masked after the product; V's rows are
// zeroed in shared memory (a zero weight times a NaN is not zero). Every wait
// is bounded; on expiry the kernel records a timeout, drains what it started
// and frees its tensor memory.
#include <climits>

#include "internal.h"
#include "prompt_common.cuh"
#include "packed_math.cuh"
#include "tcgen05.cuh"

namespace pa {

namespace {

constexpr int kM = 128;              // rows of a row tile: tensor-memory lanes
constexpr int kTile = 128;           // context tokens per K/V tile
constexpr int kMaxSlots = 13;        // of the ring of K and V tiles, in the order the products take them
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kKWarp = 9, kVWarp = 11;
constexpr int kSegs = 3;             // published segments in flight
constexpr int kSegReaders = 11;      // MMA warp, two K warps, eight softmax warps
constexpr float kSlack = 8.f;        // base-2 headroom before the running maximum moves
// Weights are 2^(s * scale - m), the product not rounded, where m is the rounded product of a largest score: its
// rounding moves all of a row's weights by one factor, which cancels: at most 2^4 up to this size of m. Beyond, the
// factor would leave fp16's range, but there different fp32 scores are 8 or more apart (in base 2), more so the
// rounding of their sums: such rows take the scale rounded up to a power of two, whose products are exact.
constexpr float kHugeScore = 134217728.f;   // 2^27
constexpr int kMaxTail = 160;        // units of a partial wave: fewer than CTAs
// p.tail_info: units of the cut wave, then eight ints a unit: first query token, query tokens, KV head, first
// head, heads, first and last CTA that holds a piece of it
constexpr int kTailUnits = 8, kTailInts = kTailUnits + 8 * kMaxTail;
constexpr int kMinPiece = 4;         // tiles a CTA takes of a cut wave, at least
// What a cut wave's pieces cost (written and read again, up to 128 KB each at head_dim 128), in tiles of its
// length: one for every so many pieces. Measured over 8 to 352 units of 8 to 128 tiles, both head dims: cuts
// by this rule run at 0.95 (U 272, 128 tiles) to 4 times (U 8) the speed of uncut waves, most of them above 1.
template <bool kTwoTiles>
constexpr int kPiecesPerTile = kTwoTiles ? 10 : 6;

template <int D, bool kTwoTiles>
struct Cfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kGroupsQ = kTwoTiles ? 2 : 1;      // row tiles of a unit
    static constexpr int kQBytes = kHalves * kM * 128;      // one row tile
    static constexpr int kSlotBytes = kHalves * kTile * 128;
    static constexpr int kRingOff = kGroupsQ * kQBytes;
    static constexpr int kSlots = ((kTwoTiles ? 224 : 220) * 1024 - kRingOff) / kSlotBytes;   // as many as fit
    static_assert(kSlots >= 5 && kSlots <= kMaxSlots, "ring");
    static constexpr int kBarOff = kRingOff + kSlots * kSlotBytes;
    // Place in the ring's order of tile i of a segment's n. Two row tiles: K0 V0 K1 V1 ...;
    // one, whose first two score tiles come before any weights: K0 K1 V0 K2 V1 ... V(n-1).
    __device__ static int k_fill(int i) { return kTwoTiles ? 2 * i : i == 0 ? 0 : 2 * i - 1; }
    __device__ static int v_fill(int i, int n) { return kTwoTiles || i == n - 1 ? 2 * i + 1 : 2 * i + 2; }
};

// One piece of a unit: K/V tiles [t0, t0 + n) of rows of one KV head.
struct Seg {
    int b, q0;            // sequence; first query token of the unit (in the batch)
    int tok0, ntok;       // the same within the sequence; query tokens of the unit
    int ctx, past;        // context tokens; PrefillSeq::past
    int kvh, h0, nh;      // KV head; first query head of its group, heads here
    int t0, n;
    int cnt[2];           // tiles each softmax group takes
    int piece;            // workspace slot, -1: the whole unit (final output), -2: no more work
};

struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];  // K: one arrival of each K warp; V: two of its warp
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2][2], o_full[2], o_free[2];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t v_land;                       // the copies of a V tile that is to be mended before it counts as full
    uint64_t join_full[2][2];              // one row tile: [segment parity][group] maxima and sums are posted
    uint64_t done;
    uint32_t tmem;
    int abort_flag;
    int last_fill[kMaxSlots], q_issued, lands;   // what has been started, for the drain after a timeout
    Seg seg[kSegs];
    int tail_prefix[kMaxTail + 1];         // tiles of the cut wave's units, summed
    int tail_work[kMaxTail];
};
struct SharedJoin {                        // one row tile, two groups: their maxima and sums
    float m[2][2][kM], l[2][2][kM];        // [segment parity][group][row]
};

template <int D, bool kTwoTiles>
constexpr size_t smem_bytes() {
    return 1024 + Cfg<D, kTwoTiles>::kBarOff + sizeof(Shared) + (kTwoTiles ? 0 : sizeof(SharedJoin));
}
static_assert(smem_bytes<128, true>() <= 227 * 1024 && smem_bytes<128, false>() <= 227 * 1024, "shared memory of a CTA");

// A whole warp waits.
__device__ __forceinline__ bool wait_bar(const PrefillParams &p, Shared *sh, uint64_t *bar, uint32_t parity) {
    return mbar_wait_warp(smem_addr(bar), parity, p.status, &sh->abort_flag);
}

// The same for a single thread (the MMA issuer inside a segment).
__device__ __forceinline__ bool wait_bar_one(const PrefillParams &p, Shared *sh, uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(smem_addr(bar), parity)) return true;
    if (*reinterpret_cast<volatile int *>(&sh->abort_flag)) return false;
    if (mbar_wait(smem_addr(bar), parity)) return true;
    record_status(p.status, kStatusTimeout);
    *reinterpret_cast<volatile int *>(&sh->abort_flag) = 1;
    return false;
}

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// D[tmem] (+)= A[tmem] * B[smem], 16-bit A packed two to a column.
__device__ __forceinline__ void tc_mma_16bit_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Warp-wide: 128 consecutive fp32 columns of this warp's 32 lanes, one wait (in
// the same block, so that no use is scheduled before it).
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
    uint32_t r[128];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"
        "}, [%128];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127"
        "}, [%129];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
          "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
          "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
          "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
          "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
          "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
          "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
          "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
          "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(taddr), "r"(taddr + 64)
        : "memory");
#pragma unroll
    for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// 32 bytes of a row, a whole sector, in one store where out allows (it is 16-byte aligned at least). Every lane
// writes a row of its own, a line a cycle: with 16-byte stores a unit's epilogue took 4,500 cycles of its 55,000
// (four prompts of 4,100 tokens 392 -> 379 us). Lanes that trade sectors first and write whole lines: no better.
__device__ __forceinline__ void store_32_bytes(void *dst, const uint32_t (&w)[8]) {
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
        return;
    }
    uint4 *d = reinterpret_cast<uint4 *>(dst);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    if constexpr (kF16) return pack_f16x2(a, b);
    else return pack_bf16x2(a, b);
}

// The largest (kMax) or smallest of a row's scores, three operands at a time.
template <bool kMax>
__device__ __forceinline__ float best3(float a, float b, float c) {
    float r;
    if constexpr (kMax) asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    else asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <bool kMax>
__device__ __forceinline__ float row_max(const float (&s)[kTile]) {
    float a[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) a[c] = s[c];
#pragma unroll
    for (int c = 4; c + 8 <= kTile; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = best3<kMax>(a[e], s[c + 2 * e], s[c + 2 * e + 1]);
    // (kTile - 4) % 8 == 4 scores are left
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = best3<kMax>(a[e], s[kTile - 4 + e], a[e]);
    return best3<kMax>(best3<kMax>(a[0], a[1], a[2]), a[3], a[3]);
}

// The power of two above |x| (x normal), with x's sign.
__device__ __forceinline__ float power_above(float x) {
    return 2.f * __uint_as_float(__float_as_uint(x) & 0xff800000u);
}

// Tiles a unit (row tiles from token tok0 of the sequence) has to visit.
__device__ __forceinline__ int unit_tiles(const PrefillParams &p, const PrefillSeq &s, int tile) {
    const int last = min((tile + 1) * p.tile_tokens, s.qlen) - 1;
    return (prefill_sees(p, s, last) + kTile - 1) / kTile;
}

// ---------------------------------------------------------------------------
// The schedule (one warp): segments of this CTA, in order.
// ---------------------------------------------------------------------------
struct Scheduler {           // (the host keeps the batch's units below 2^31)
    int units, nfull;        // all units; units taken whole
    int next;                // next whole unit of this CTA (lane 0 where they are drawn from p.counter)
    int tail, a, e;          // units of the cut wave; this CTA's remaining range of its tiles
    int r;                   // unit of the cut wave that holds tile a
    // 32 sequences at a time, one a lane: its extent, its row tiles and those before it in the chunk
    int base, before, total; // first sequence of the chunk, row tiles before the chunk, row tiles in it
    int b;                   // this lane's sequence (p.order: longest contexts first)
    PrefillSeq seq;
    int n, excl;
};

// The cut wave's tiles over the CTAs that share it: the first tiles % ctas take one more.
__device__ __forceinline__ int range_begin(int c, int tiles, int ctas) { return c * (tiles / ctas) + min(c, tiles % ctas); }
__device__ __forceinline__ int range_owner(int x, int tiles, int ctas) {
    const int q = tiles / ctas, more = tiles % ctas, edge = more * (q + 1);
    return x < edge ? x / (q + 1) : more + (x - edge) / q;   // (q >= 1: every CTA has a tile)
}

__device__ __forceinline__ void sched_chunk(const PrefillParams &p, Scheduler &sc, int lane) {
    sc.b = sc.base + lane;
    sc.seq = PrefillSeq{0, 0, 0, 0};
    if (sc.b < p.num_seqs) {
        if (p.order) sc.b = p.order[sc.b];
        sc.seq = prefill_seq(p, sc.b);
    }
    sc.n = (sc.seq.qlen + p.tile_tokens - 1) / p.tile_tokens;
    int sum = sc.n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    sc.excl = sum - sc.n;
    sc.total = __shfl_sync(0xffffffffu, sum, 31);
}

template <bool kTwoTiles>
__device__ void sched_init(const PrefillParams &p, Shared *sh, Scheduler &sc, int lane) {
    const int ys = p.num_kv_heads * p.ntile;
    const int ctas = gridDim.x;
    int rows = 0;
    for (sc.base = 0; sc.base < p.num_seqs; sc.base += 32) {
        sched_chunk(p, sc, lane);
        rows += sc.total;
    }
    sc.units = sc.nfull = rows * ys;
    sc.next = blockIdx.x;
    sc.tail = sc.r = sc.a = sc.e = 0;
    const int rem = sc.units % ctas;
    // (a query_start that breaks its contract may describe more units than the workspace was sized for)
    if (p.nsplit > 1 && rem > 0 && rem <= p.max_tail) {
        sc.nfull = sc.units - rem;
        sc.tail = rem;
        // tiles of the tail's row tiles [x_lo, x_hi], lanes over sequences
        const int x_lo = sc.nfull / ys, x_hi = (sc.units - 1) / ys;
        int before = 0;
        for (sc.base = 0; sc.base < p.num_seqs; sc.base += 32) {
            if (p.num_seqs > 32) sched_chunk(p, sc, lane);
            const int first = before + sc.excl;                    // this sequence's row tiles: first .. first + n - 1
            for (int t = max(first, x_lo); t <= min(first + sc.n - 1, x_hi); ++t)
                sh->tail_work[t - x_lo] = max(1, unit_tiles(p, sc.seq, sc.n - 1 - (t - first)));
            before += sc.total;
        }
        __syncwarp();
        // lane l holds units [l per, (l + 1) per): their tiles
        const int per = (sc.tail + 31) / 32, skip = sc.nfull - x_lo * ys, r0 = lane * per;
        constexpr int kPer = (kMaxTail + 31) / 32;
        int w[kPer], mine = 0, most = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            w[i] = i < per && r0 + i < sc.tail ? sh->tail_work[(skip + r0 + i) / ys] : 0;
            mine += w[i];
            most = max(most, w[i]);
        }
        const int tiles = __reduce_add_sync(0xffffffffu, mine);
        most = __reduce_max_sync(0xffffffffu, most);
        // the shortest length to which units can be cut with one piece a CTA
        auto pieces = [&](int len) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) n += (w[i] + len - 1) / len;
            return n;
        };
        const int even = (tiles + ctas - 1) / ctas;
        int len = max(even, kMinPiece), hi = max(most, len);       // (the units themselves are at most ctas)
        while (len < hi) {
            const int mid = (len + hi) / 2;
            if (static_cast<int>(__reduce_add_sync(0xffffffffu, pieces(mid))) <= ctas) hi = mid;
            else len = mid + 1;
        }
        // tiles saved, less what the pieces cost: units cut into pieces, one a CTA, or equal ranges of tiles that
        // run across units (shorter, but up to two more pieces a CTA), or neither
        const int cuts_all = __reduce_add_sync(0xffffffffu, pieces(len));
        const int by_pieces = most - len - (cuts_all > sc.tail ? cuts_all : 0) / kPiecesPerTile<kTwoTiles>,
                  by_ranges = most - even - (sc.tail + ctas) / kPiecesPerTile<kTwoTiles>;
        const bool ranges = by_ranges > by_pieces;
        if (max(by_ranges, by_pieces) <= 0) {
            sc.nfull = sc.units;
            sc.tail = 0;
        } else {
            const int tail_ctas = max(1, min(ctas, tiles / kMinPiece)), c = blockIdx.x;
            if (ranges && c < tail_ctas) {
                sc.a = range_begin(c, tiles, tail_ctas);
                sc.e = range_begin(c + 1, tiles, tail_ctas);
            }
            const int cuts = pieces(len);
            int at = mine, first = cuts;                           // tiles, pieces before this lane's units
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, at, d), q = __shfl_up_sync(0xffffffffu, first, d);
                if (lane >= d) {
                    at += o;
                    first += q;
                }
            }
            at -= mine;
            first -= cuts;
            int holds = -1, a = 0, e = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (w[i] == 0) continue;
                const int r = r0 + i, n = (w[i] + len - 1) / len, j = c - first;
                sh->tail_prefix[r] = at;
                if (ranges ? at <= sc.a && sc.a < at + w[i] : j >= 0 && j < n) {   // holds this CTA's (first) piece
                    holds = r;
                    if (!ranges) {
                        a = at + range_begin(j, w[i], n);
                        e = at + range_begin(j + 1, w[i], n);
                    }
                }
                if (c == 0) {                                      // for the merge
                    int *d = p.tail_info + kTailUnits + r * 8;
                    d[5] = ranges ? range_owner(at, tiles, tail_ctas) : first;
                    d[6] = ranges ? range_owner(at + w[i] - 1, tiles, tail_ctas) : first + n - 1;
                }
                at += w[i];
                first += n;
            }
            if (lane == 0) sh->tail_prefix[sc.tail] = tiles;
            const unsigned who = __ballot_sync(0xffffffffu, holds >= 0);
            if (who) {
                const int l = __ffs(who) - 1;
                sc.r = __shfl_sync(0xffffffffu, holds, l);
                if (!ranges) {
                    sc.a = __shfl_sync(0xffffffffu, a, l);
                    sc.e = __shfl_sync(0xffffffffu, e, l);
                }
            }
            __syncwarp();
        }
    }
    sc.base = sc.before = 0;
    if (p.num_seqs > 32) sched_chunk(p, sc, lane);
    if (blockIdx.x == 0 && p.nsplit > 1 && lane == 0) p.tail_info[0] = sc.tail;   // for the merge
}

// The next segment of this CTA into g (lane 0 writes it).
template <bool kTwoTiles>
__device__ __forceinline__ void sched_next(const PrefillParams &p, Shared *sh, Scheduler &sc, Seg &g, int lane) {
    const int ys = p.num_kv_heads * p.ntile;
    int u, t0 = 0, t1 = INT_MAX, piece = -1;
    if (const int mine = __shfl_sync(0xffffffffu, sc.next, 0); mine < sc.nfull) {
        u = mine;
        // the next one is drawn now and waited for at the next call
        if (!p.counter) sc.next += gridDim.x;
        else if (lane == 0) sc.next = gridDim.x + atomicAdd(p.counter, 1);
    } else if (sc.a < sc.e) {
        while (sh->tail_prefix[sc.r + 1] <= sc.a) ++sc.r;
        const int p0 = sh->tail_prefix[sc.r], p1 = sh->tail_prefix[sc.r + 1];
        u = sc.nfull + sc.r;
        t0 = sc.a - p0;
        t1 = min(sc.e, p1) - p0;
        if (t0 > 0 || t1 < p1 - p0) piece = static_cast<int>(blockIdx.x) + sc.r;
        sc.a = p0 + t1;
    } else {
        if (lane == 0) g.piece = -2;
        return;
    }
    // the sequence whose row tiles hold u / ys (never before the chunk: units only go up)
    const int x = u / ys;
    while (x >= sc.before + sc.total && sc.base + 32 < p.num_seqs) {
        sc.before += sc.total;
        sc.base += 32;
        sched_chunk(p, sc, lane);
    }
    const unsigned hit = __ballot_sync(0xffffffffu, x < sc.before + sc.excl + sc.n);
    const int l = hit ? __ffs(hit) - 1 : 31;
    PrefillSeq s;
    s.q0 = __shfl_sync(0xffffffffu, sc.seq.q0, l);
    s.qlen = __shfl_sync(0xffffffffu, sc.seq.qlen, l);
    s.ctx = __shfl_sync(0xffffffffu, sc.seq.ctx, l);
    s.past = __shfl_sync(0xffffffffu, sc.seq.past, l);
    const int ntiles = __shfl_sync(0xffffffffu, sc.n, l), b = __shfl_sync(0xffffffffu, sc.b, l);
    const int from = x - sc.before - __shfl_sync(0xffffffffu, sc.excl, l);
    if (lane != 0) return;
    // within a sequence the last row tile first: the longest work of a causal mask starts first
    const int tile = ntiles - 1 - from, y = u - x * ys;
    const int row_tokens = kTwoTiles ? p.tile_tokens / 2 : p.tile_tokens;
    g.b = b;
    g.tok0 = tile * p.tile_tokens;
    g.q0 = s.q0 + g.tok0;
    g.ntok = min(p.tile_tokens, s.qlen - g.tok0);
    g.ctx = s.ctx;
    g.past = s.past;
    g.kvh = y / p.ntile;
    g.h0 = (y - g.kvh * p.ntile) * p.heads_per_tile;
    g.nh = min(p.heads_per_tile, p.group - g.h0);
    const int tiles = unit_tiles(p, s, tile);
    g.t0 = t0;
    g.n = max(0, min(t1, tiles) - t0);
    if (kTwoTiles) {   // the first row tile may see one K/V tile fewer, the second may have no tokens
        const int first = (prefill_sees(p, s, g.tok0 + min(row_tokens, g.ntok) - 1) + kTile - 1) / kTile;
        g.cnt[0] = max(0, min(g.n, first - t0));
        g.cnt[1] = g.ntok > row_tokens ? g.n : 0;
    } else {
        g.cnt[0] = (g.n + 1) / 2;
        g.cnt[1] = g.n / 2;
    }
    g.piece = piece;
    if (piece >= 0 && t0 == 0) {   // a cut unit, for the merge
        int *d = p.tail_info + kTailUnits + sc.r * 8;
        d[0] = g.q0;
        d[1] = g.ntok;
        d[2] = g.kvh;
        d[3] = g.h0;
        d[4] = g.nh;
    }
}

// Tokens of one TMA box: a cache block, at most 64.
__device__ __forceinline__ int box_tokens(const PrefillParams &p) {
    return p.contig_stride > 0 ? 64 : min(p.block_size, 64);
}

// The ids of the blocks a producer warp is about to load, 32 at a time.
struct BlockIds {
    int first;     // block index of lane 0's entry; -1: nothing loaded
    int id;
};
__device__ __forceinline__ int block_id(const PrefillParams &p, BlockIds &c, int b, int blk, int nblk, int lane) {
    if (c.first < 0 || blk < c.first || blk >= c.first + 32) {
        c.first = blk;
        const int e = blk + lane;
        c.id = e < nblk ? p.block_tables[static_cast<int64_t>(b) * p.max_blocks + e] : -1;
    }
    return __shfl_sync(0xffffffffu, c.id, blk - c.first);
}

template <int D, bool kTwoTiles, bool kF16, bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
prefill_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                  const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ PrefillParams p) {
    using C = Cfg<D, kTwoTiles>;
    constexpr int kSlots = C::kSlots;
    // V in shared memory. kWide (boxes of 32 tokens or more): [half][token][128 bytes], one box a half. Else
    // (16 or 8, half as many boxes): boxes of [half][token][128 bytes] one after another. In either the
    // 16-token steps of the products are a constant apart, which the MMA issue depends on.
    constexpr int kVBoxHalves = kWide ? 1 : C::kHalves;
    constexpr int kVStep = kVBoxHalves * 16 * 128;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *q_s = smem, *ring = smem + C::kRingOff;
    Shared *sh = reinterpret_cast<Shared *>(smem + C::kBarOff);
    SharedJoin *join = reinterpret_cast<SharedJoin *>(sh + 1);   // one row tile only
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    if (warp == kVWarp && lane == 0) {
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_addr(&sh->full[i]), 2);
            mbar_init(smem_addr(&sh->empty[i]), 1);
            sh->last_fill[i] = -1;
        }
        mbar_init(smem_addr(&sh->q_full), 1);
        mbar_init(smem_addr(&sh->q_empty), 1);
        for (int g = 0; g < 2; ++g) {
            mbar_init(smem_addr(&sh->s_full[g]), 1);
            mbar_init(smem_addr(&sh->p_full[g][0]), 4);
            mbar_init(smem_addr(&sh->p_full[g][1]), 4);
            mbar_init(smem_addr(&sh->o_full[g]), 1);
            mbar_init(smem_addr(&sh->o_free[g]), kTwoTiles ? 4 : 8);
            mbar_init(smem_addr(&sh->join_full[0][g]), 4);
            mbar_init(smem_addr(&sh->join_full[1][g]), 4);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(smem_addr(&sh->seg_full[i]), 1);
            mbar_init(smem_addr(&sh->seg_empty[i]), kSegReaders);
        }
        mbar_init(smem_addr(&sh->done), 1);
        mbar_init(smem_addr(&sh->v_land), 1);
        sh->abort_flag = 0;
        sh->q_issued = sh->lands = 0;
        mbar_fence_init();
    } else if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&sh->tmem), 512u);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(sh->tmem);
    grid_dependency_wait();
    // tensor-memory columns: S of group g at 128 g, P in its place, O at 256 + 128 g
    auto s_col = [&](int g) { return tmem + g * 128; };
    auto o_col = [&](int g) { return tmem + 256 + g * 128; };
    const int R = box_tokens(p), r_shift = 31 - __clz(R);                    // powers of two, like the block size
    const int bs_shift = 31 - __clz(p.block_size);

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kVWarp) {
            // ---------------- the schedule, Q and V ----------------
            Scheduler sc;
            sched_init<kTwoTiles>(p, sh, sc, lane);
            const uint64_t policy = l2_policy_evict_normal(), q_policy = l2_policy_evict_first();
            const int q_tokens = kTwoTiles ? p.tile_tokens / 2 : p.tile_tokens;
            // segment k's readers have all begun it before segment k + kSegs takes its place
            auto publish = [&](int k) {
                if (k >= kSegs && !wait_bar(p, sh, &sh->seg_empty[k % kSegs], ((k / kSegs) - 1) & 1)) return false;
                sched_next<kTwoTiles>(p, sh, sc, sh->seg[k % kSegs], lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh->seg_full[k % kSegs]));
                return true;
            };
            int fills = 0, lands = 0;            // of the segments before: ring tiles, mended V tiles
            publish(0);
            for (int k = 0;; ++k) {
                const Seg *g = &sh->seg[k % kSegs];
                if (g->piece == -2) break;
                if (k > 0 && !wait_bar(p, sh, &sh->q_empty, (k - 1) & 1)) break;
                const int b = uniform(g->b), ctx = uniform(g->ctx), kvh = uniform(g->kvh), n = uniform(g->n),
                          first = uniform(g->t0), h0 = uniform(g->h0), q0 = uniform(g->q0);
                const uint32_t qf = smem_addr(&sh->q_full);
                if (elect_one()) {
                    mbar_arrive_expect_tx(qf, static_cast<uint32_t>(C::kGroupsQ * C::kHalves * q_tokens *
                                                                    p.heads_per_tile * 128));
                    // (dim, half, head in group, KV head, token): rows token * heads_per_tile + head
#pragma unroll
                    for (int t = 0; t < C::kGroupsQ; ++t)
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            tma_load_5d(smem_addr(q_s + t * C::kQBytes + h * (kM * 128)), &tmap_q, 0, h, h0, kvh,
                                        q0 + t * q_tokens, qf, q_policy);
                    sh->q_issued = k + 1;
                }
                __syncwarp();
                // the K warps run into the next segment while this one's V still comes
                if (!publish(k + 1)) break;
                BlockIds ids{-1, 0};
                const int nblk = (ctx + p.block_size - 1) >> bs_shift;
                bool ok = true;
                for (int i = 0; i < n; ++i) {
                    const int f = fills + C::v_fill(i, n), slot = f % kSlots, t0 = (first + i) * kTile;
                    if (f >= kSlots && !wait_bar(p, sh, &sh->empty[slot], ((f / kSlots) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const int boxes = (min(ctx - t0, kTile) + R - 1) >> r_shift, valid = ctx - t0;
                    const uint32_t full = smem_addr(&sh->full[slot]);
                    // where the context ends inside the tile, its copies land on a barrier of this warp's own
                    const bool mend = valid < kTile;
                    const uint32_t land = mend ? smem_addr(&sh->v_land) : full;
                    const uint32_t dst = smem_addr(ring + slot * C::kSlotBytes);
                    if (elect_one()) {
                        mbar_arrive_expect_tx(land, static_cast<uint32_t>(boxes * C::kHalves * R * 128));
                        if (mend) {
                            sh->lands = lands + 1;
                        } else {
                            mbar_arrive(full);
                            sh->last_fill[slot] = f;
                        }
                    }
                    __syncwarp();
                    for (int j = 0; j < boxes; ++j) {
                        const int tok = t0 + j * R;
                        int at = tok, blk = 0;
                        if (p.contig_stride > 0) {
                            at += b * p.contig_stride;
                        } else {
                            blk = block_id(p, ids, b, tok >> bs_shift, nblk, lane);
                            at = tok & (p.block_size - 1);
                        }
                        if (elect_one()) {
#pragma unroll
                            for (int h = 0; h < C::kHalves; h += kVBoxHalves)
                                tma_load_5d(dst + h * (kTile * 128) + j * (kVBoxHalves * R * 128), &tmap_v, 0, at, h, kvh, blk,
                                            land, policy);
                        }
                        __syncwarp();
                    }
                    if (mend) {   // zero the rows past the context; then the tile is full
                        if (!wait_bar(p, sh, &sh->v_land, lands & 1)) {
                            ok = false;
                            break;
                        }
                        ++lands;
                        unsigned char *v = ring + slot * C::kSlotBytes;
                        for (int x = lane; x < (kTile - valid) * C::kHalves * 8; x += 32) {
                            const int row = valid + x / (C::kHalves * 8), c = x % (C::kHalves * 8);
                            const int at = kWide ? (c / 8) * (kTile * 128) + row * 128
                                                 : (row >> r_shift) * (C::kHalves * R * 128) + (c / 8) * (R * 128) + (row & (R - 1)) * 128;
                            *reinterpret_cast<uint4 *>(v + at + (c % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(full);
                            mbar_arrive(full);
                        }
                    }
                }
                if (!ok) break;
                fills += 2 * n;
            }
        } else if (warp != kMmaWarp) {
            // ---------------- K, 64 tokens of every tile ----------------
            const int part = warp - kKWarp;
            const uint64_t policy = l2_policy_evict_normal();
            int fills = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const Seg *g = &sh->seg[k % kSegs];
                if (!wait_bar(p, sh, &sh->seg_full[k % kSegs], (k / kSegs) & 1) || g->piece == -2) break;
                const int b = uniform(g->b), ctx = uniform(g->ctx), kvh = uniform(g->kvh), n = uniform(g->n),
                          first = uniform(g->t0);
                if (lane == 0) mbar_arrive(smem_addr(&sh->seg_empty[k % kSegs]));
                const int nblk = (ctx + p.block_size - 1) >> bs_shift;
                BlockIds ids{-1, 0};
                for (int i = 0; i < n; ++i) {
                    const int f = fills + C::k_fill(i), slot = f % kSlots, t0 = (first + i) * kTile + part * 64;
                    if (f >= kSlots && !wait_bar(p, sh, &sh->empty[slot], ((f / kSlots) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const int boxes = max(0, min(ctx - t0, 64) + R - 1) >> r_shift;
                    const uint32_t full = smem_addr(&sh->full[slot]);
                    const uint32_t dst = smem_addr(ring + slot * C::kSlotBytes) + part * 64 * 128;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(full, static_cast<uint32_t>(boxes * C::kHalves * R * 128));
                        sh->last_fill[slot] = f;
                    }
                    __syncwarp();
                    for (int j = 0; j < boxes; ++j) {
                        const int tok = t0 + j * R;
                        int at = tok, blk = 0;
                        if (p.contig_stride > 0) {
                            at += b * p.contig_stride;
                        } else {
                            blk = block_id(p, ids, b, tok >> bs_shift, nblk, lane);
                            at = tok & (p.block_size - 1);
                        }
                        if (elect_one()) {
#pragma unroll
                            for (int h = 0; h < C::kHalves; ++h)
                                tma_load_5d(dst + h * (kTile * 128) + j * (R * 128), &tmap_k, 0, at, h, kvh, blk, full,
                                            policy);
                        }
                        __syncwarp();
                    }
                }
                fills += 2 * n;
            }
        } else {
            // ---------------- MMA issue ----------------
            constexpr uint32_t id_qk = idesc_16bit_f32(kM, kTile, false, false, kF16);
            constexpr uint32_t id_pv = idesc_16bit_f32(kM, D, false, true, kF16);
            const uint64_t q_desc = smem_desc_sw128(smem_addr(q_s), 16, 1024), k_desc = smem_desc_sw128(smem_addr(ring), 16, 1024);
            const uint64_t v_desc = smem_desc_sw128(smem_addr(ring), kWide ? kTile * 128 : R * 128, kWide || R >= 16 ? 1024 : C::kHalves * 1024);
            int fills = 0;                       // ring tiles of the segments before
            int s_cnt[2] = {0, 0}, o_cnt[2] = {0, 0};   // a group's tiles; its segments with any
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const Seg *g = &sh->seg[k % kSegs];
                if (!wait_bar(p, sh, &sh->seg_full[k % kSegs], (k / kSegs) & 1) || g->piece == -2) break;
                const int n = uniform(g->n);
                const int cnt[2] = {uniform(g->cnt[0]), uniform(g->cnt[1])};
                if (lane == 0) mbar_arrive(smem_addr(&sh->seg_empty[k % kSegs]));
                if (!wait_bar(p, sh, &sh->q_full, k & 1)) break;
                // places in the ring: the next K and V tile's slot and phase, stepped along
                struct Place {
                    int slot, phase;
                    __device__ __forceinline__ void step(int by) {
                        slot += by;
                        if (slot >= kSlots) {
                            slot -= kSlots;
                            phase ^= 1;
                        }
                    }
                };
                auto wait_at = [&](const Place &at) { return wait_bar_one(p, sh, &sh->full[at.slot], at.phase); };
                // the slot is free once every product issued so far has run
                auto release = [&](const Place &at) { tc_commit(smem_addr(&sh->empty[at.slot])); };
                auto issue_s = [&](int grp, const Place &at) {
                    tc_fence_after();
                    const uint64_t qd = q_desc + (kTwoTiles ? grp : 0) * desc_step(C::kQBytes);
                    const uint64_t kd = k_desc + static_cast<uint32_t>(at.slot) * static_cast<uint32_t>(C::kSlotBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int half = kk / 4, off = (kk % 4) * 32;
                        tc_mma_16bit(s_col(grp), qd + desc_step(half * (kM * 128) + off),
                                     kd + desc_step(half * (kTile * 128) + off), id_qk, kk > 0 ? 1u : 0u);
                    }
                    tc_commit(smem_addr(&sh->s_full[grp]));
                };
                // O += P V of the group's tile j, in two halves of 64 tokens as their weights appear
                auto issue_pv = [&](int grp, int j, const Place &at) {
                    const uint64_t vd = v_desc + static_cast<uint32_t>(at.slot) * static_cast<uint32_t>(C::kSlotBytes >> 4);
                    if (j == 0 && o_cnt[grp] > 0 && !wait_bar_one(p, sh, &sh->o_free[grp], (o_cnt[grp] - 1) & 1)) return false;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!wait_bar_one(p, sh, &sh->p_full[grp][h], (s_cnt[grp] + j) & 1)) return false;
                        tc_fence_after();
#pragma unroll
                        for (int kk = h * 4; kk < h * 4 + 4; ++kk)
                            tc_mma_16bit_ts(o_col(grp), s_col(grp) + kk * 8, vd + desc_step(kk * kVStep), id_pv,
                                            (j > 0 || kk > 0) ? 1u : 0u);
                    }
                    if (j == cnt[grp] - 1) tc_commit(smem_addr(&sh->o_full[grp]));
                    return true;
                };
                // the products of one segment, issued by one thread: K and V are waited for ahead of the
                // weights, so that nothing stands between a group's P V and its next S
                auto segment = [&]() {
                    if (n == 0) {
                        tc_commit(smem_addr(&sh->q_empty));
                        return true;
                    }
                    Place kp{fills % kSlots, (fills / kSlots) & 1}, vp = kp;
                    if constexpr (kTwoTiles) {
                        if (!wait_at(kp)) return false;
                        if (cnt[0] > 0) issue_s(0, kp);
                        if (cnt[1] > 0) issue_s(1, kp);
                        release(kp);
                        if (n == 1) tc_commit(smem_addr(&sh->q_empty));
                        vp.step(1);
                        kp.step(2);
                        for (int i = 0; i < n; ++i) {
                            if (!wait_at(vp) || (i + 1 < n && !wait_at(kp))) return false;
                            if (i < cnt[0] && !issue_pv(0, i, vp)) return false;
                            if (i + 1 < cnt[0]) issue_s(0, kp);
                            if (i < cnt[1] && !issue_pv(1, i, vp)) return false;
                            release(vp);
                            if (i + 1 < n) {
                                if (i + 1 < cnt[1]) issue_s(1, kp);
                                release(kp);
                                if (i + 2 == n) tc_commit(smem_addr(&sh->q_empty));
                            }
                            vp.step(2);
                            kp.step(2);
                        }
                    } else {
                        for (int i = 0; i < 2 && i < n; ++i) {
                            if (!wait_at(kp)) return false;
                            issue_s(i, kp);
                            release(kp);
                            if (i == n - 1) tc_commit(smem_addr(&sh->q_empty));
                            kp.step(i == 0 ? 1 : 2);
                        }
                        vp.step(n == 1 ? 1 : 2);
                        for (int i0 = 0; i0 < n; i0 += 2) {
#pragma unroll
                            for (int grp = 0; grp < 2; ++grp) {
                                const int i = i0 + grp;
                                if (i >= n) break;
                                if (!wait_at(vp) || (i + 2 < n && !wait_at(kp)) ||
                                    !issue_pv(grp, i0 >> 1, vp))
                                    return false;
                                release(vp);
                                if (i + 2 < n) {
                                    issue_s(grp, kp);
                                    release(kp);
                                    if (i + 3 == n) tc_commit(smem_addr(&sh->q_empty));
                                }
                                vp.step(i + 2 < n ? 2 : 1);
                                kp.step(2);
                            }
                        }
                    }
                    return true;
                };
                bool done = true;
                if (elect_one()) done = segment();
                __syncwarp();
                ok = __all_sync(0xffffffffu, done);
                fills += 2 * n;
#pragma unroll
                for (int grp = 0; grp < 2; ++grp) {
                    s_cnt[grp] += cnt[grp];
                    o_cnt[grp] += cnt[grp] > 0;
                }
            }
            // every MMA the issuing thread started has completed once `done` arrives
            if (elect_one()) {
                tc_commit(smem_addr(&sh->done));
                if (!mbar_wait(smem_addr(&sh->done), 0)) record_status(p.status, kStatusTimeout);
            }
            __syncwarp();
        }
    } else {
        // ---------------- softmax ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int grp = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int row_tokens = kTwoTiles ? p.tile_tokens / 2 : p.tile_tokens;
        const int rt = row / p.heads_per_tile, rh = row - rt * p.heads_per_tile;
        const float sl2 = p.scale_log2;
        const bool up = sl2 >= 0.f;
        int s_cnt = 0, o_cnt = 0, o_other = 0;   // tiles; segments in which this / the other group had any
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Seg *g = &sh->seg[k % kSegs];
            if (!wait_bar(p, sh, &sh->seg_full[k % kSegs], (k / kSegs) & 1) || g->piece == -2) break;
            const int cnt = g->cnt[grp], first = g->t0, piece = g->piece, q0 = g->q0;
            const int tok = (kTwoTiles ? grp * row_tokens : 0) + rt;            // query token within the unit
            const bool live = rt < row_tokens && tok < g->ntok && rh < g->nh;
            // rows that are not there need no masking but the context's end: their outputs are never stored
            const int sees = !live || !p.causal ? g->ctx : max(0, min(g->ctx, g->past + g->tok0 + tok + 1));
            const int64_t orow = static_cast<int64_t>(q0 + tok) * p.num_heads + g->kvh * p.group + g->h0 + rh;
            const int other = kTwoTiles ? 0 : g->cnt[grp ^ 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh->seg_empty[k % kSegs]));
            const int whole = __reduce_min_sync(0xffffffffu, sees);             // every row of the warp sees these tokens
            float m = kLowestScore, l = 0.f;
            float mul = sl2;             // (see kHugeScore)
            for (int j = 0; j < cnt; ++j) {
                if (!wait_bar(p, sh, &sh->s_full[grp], s_cnt & 1)) { ok = false; break; }
                ++s_cnt;
                tc_fence_after();
                const int t0 = (first + (kTwoTiles ? j : 2 * j + grp)) * kTile;
                float s[kTile];
                tmem_ld128(s_col(grp) + lanes, s);
                if (t0 + kTile > whole) {     // (the scale is never zero: infinity times it is the mask)
                    const int valid = sees - t0;
                    const float never = up ? -INFINITY : INFINITY;
#pragma unroll
                    for (int c = 0; c < kTile; ++c) s[c] = c < valid ? s[c] : never;
                }
                uint64_t sum[2] = {0, 0};
                auto weights = [&](int half) {   // 2^(s * scale - m), two at a time
                    const uint64_t mul2 = pair(mul, mul), neg2 = pair(-m, -m);
#pragma unroll
                    for (int c0 = half * 64; c0 < half * 64 + 64; c0 += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            float e0, e1;
                            unpair(fma2(pair(s[c0 + 2 * c], s[c0 + 2 * c + 1]), mul2, neg2), e0, e1);
                            e0 = fast_exp2(e0);
                            e1 = fast_exp2(e1);
                            sum[c & 1] = add2(sum[c & 1], pair(e0, e1));
                            w[c] = pack16<kF16>(e0, e1);   // the weights' one rounding, to the caches' type
                        }
                        tmem_st16_nowait(s_col(grp) + lanes + c0 / 2, w);
                    }
                };
                auto hand_over = [&](int half) {   // 64 tokens' weights are there: the products may start on them
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh->p_full[grp][half]));
                };
                const float top = up ? row_max<true>(s) : row_max<false>(s), mx = top * mul;
                const bool need = mx > m + kSlack;
                if (__any_sync(0xffffffffu, need)) {
                    if (need) mul = fabsf(top * sl2) > kHugeScore ? power_above(sl2) : sl2;
                    const float m_new = need ? top * mul : m, alpha = fast_exp2(m - m_new);
                    m = m_new;
                    l *= alpha;
                    // S of this tile was issued behind the group's previous P V: O is at rest until P appears
#pragma unroll 1
                    for (int c = 0; c < D && j > 0; c += 16) {
                        float o[16];
                        uint32_t w[16];
                        tmem_ld16(o_col(grp) + lanes + c, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
                        tmem_st16_nowait(o_col(grp) + lanes + c, w);
                    }
                    tmem_wait_st();
                }
                weights(0);
                hand_over(0);
                weights(1);
                hand_over(1);
                float a0, a1;
                unpair(add2(sum[0], sum[1]), a0, a1);
                l += a0 + a1;
            }
            if (!ok) break;
            // ---- epilogue ----
            float inv = 0.f, wa = 1.f, wb = 0.f;   // O = inv * (wa O_grp + wb O_other)
            if constexpr (!kTwoTiles) {            // the other group's share of the row
                join->m[k & 1][grp][row] = m;
                join->l[k & 1][grp][row] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh->join_full[k & 1][grp]));
                if (!wait_bar(p, sh, &sh->join_full[k & 1][grp ^ 1], (k >> 1) & 1)) break;
                const float mo = join->m[k & 1][grp ^ 1][row], lo = join->l[k & 1][grp ^ 1][row];
                const float M = fmaxf(m, mo);
                wa = cnt > 0 ? fast_exp2(m - M) : 0.f;
                wb = other > 0 ? fast_exp2(mo - M) : 0.f;
                l = (cnt > 0 ? l * wa : 0.f) + (other > 0 ? lo * wb : 0.f);
                m = M;
            }
            inv = piece >= 0 ? 1.f : l > 0.f ? 1.f / l : l;   // pieces stay unnormalised; 0: an empty row; NaN stays
            wa *= inv;
            wb *= inv;
            if (cnt > 0 && !wait_bar(p, sh, &sh->o_full[grp], o_cnt & 1)) break;
            if (!kTwoTiles && other > 0 && !wait_bar(p, sh, &sh->o_full[grp ^ 1], o_other & 1)) break;
            tc_fence_after();
            // one row tile: each group writes half of the columns, from both groups' O
            constexpr int kCols = kTwoTiles ? D : D / 2;
            const int col0 = kTwoTiles ? 0 : grp * kCols;
            // (not unrolled, few columns at a time: code that runs once a unit costs its fetch from memory; with 32
            // columns short units take 1 to 3 % longer, with the loop unrolled by two 2 to 10 %)
#pragma unroll 1
            for (int c = 0; c < kCols; c += 16) {
                float o[16];
                if (cnt > 0) {
                    tmem_ld16(o_col(grp) + lanes + col0 + c, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= wa;
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.f;
                }
                if (!kTwoTiles && other > 0) {
                    float x[16];
                    tmem_ld16(o_col(grp ^ 1) + lanes + col0 + c, x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = fmaf(x[e], wb, o[e]);
                }
                if (c + 16 == kCols) {   // O has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (cnt > 0) mbar_arrive(smem_addr(&sh->o_free[grp]));
                        if (!kTwoTiles && other > 0) mbar_arrive(smem_addr(&sh->o_free[grp ^ 1]));
                    }
                }
                if (piece >= 0) {        // [piece][row tile][column][row]: coalesced over the warp's rows
                    float *dst = p.part_out +
                                 ((static_cast<int64_t>(piece) * C::kGroupsQ + (kTwoTiles ? grp : 0)) * D + col0 + c) * kM + row;
#pragma unroll
                    for (int e = 0; e < 16; ++e) dst[e * kM] = o[e];
                } else if (live) {
                    if (p.out_type == (kF16 ? 2 : 1)) {
                        uint16_t *dst = static_cast<uint16_t *>(p.out) + orow * D + col0 + c;
                        uint32_t w[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) w[x] = pack16<kF16>(o[2 * x], o[2 * x + 1]);
                        store_32_bytes(dst, w);
                    } else if (p.out_type == 0) {
                        float *dst = static_cast<float *>(p.out) + orow * D + col0 + c;
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            uint32_t w[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) w[x] = __float_as_uint(o[e + x]);
                            store_32_bytes(dst + e, w);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) store_pair_as(p.out, p.out_type, orow * D + col0 + c + e, o[e], o[e + 1]);
                    }
                }
            }
            if (piece >= 0 && (kTwoTiles || grp == 0)) {
                const int64_t at = (static_cast<int64_t>(piece) * C::kGroupsQ + (kTwoTiles ? grp : 0)) * kM + row;
                p.part_max[at] = m;
                p.part_sum[at] = l;
            }
            if (cnt > 0) ++o_cnt;
            if (other > 0) ++o_other;
        }
    }

    // ---- drain: copies still landing (after a timeout), then the tensor memory ----
    grid_dependents_launch();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *reinterpret_cast<volatile int *>(&sh->abort_flag)) {
        // bounded: a slot of which one warp's half was never started does not complete
        for (int i = 0; i < kSlots; ++i)
            if (sh->last_fill[i] >= 0)
                mbar_wait_for(smem_addr(&sh->full[i]), (sh->last_fill[i] / kSlots) & 1, 100000000ull);
        if (sh->lands) mbar_wait_for(smem_addr(&sh->v_land), (sh->lands - 1) & 1, 100000000ull);
        if (sh->q_issued) mbar_wait_for(smem_addr(&sh->q_full), (sh->q_issued - 1) & 1, 100000000ull);
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512u);
    }
}

// ---------------------------------------------------------------------------
// Ahead of a launch whose CTAs draw their units: the counter, and the order in
// which the sequences' units are drawn, longest contexts first, so that the
// last ones are short (64 ragged chunks: 436 us in the batch's order, 415 so then; at
// head_dim 64 405 and 365; 1,000 sequences of up to 100 tokens 482 and 499, so
// only batches of at most kPrefillOrderSeqs are ordered: the CTAs go through the
// list themselves). One CTA, a thread a sequence, which counts those that go
// before its own.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPrefillOrderSeqs)
prefill_order_kernel(const __grid_constant__ PrefillParams p) {
    __shared__ alignas(16) int tiles[kPrefillOrderSeqs];
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = threadIdx.x, n = p.num_seqs;
    int mine = -1;
    if (b < n) mine = (prefill_seq(p, b).ctx + kTile - 1) / kTile;
    tiles[b] = mine;
    __syncthreads();
    if (b == 0) *p.counter = 0;
    if (b >= n) return;
    int rank = 0;
    for (int j = 0; j < n; j += 4) {   // (the block is whole warps: the entries past n are there, and -1)
        const int4 t = *reinterpret_cast<const int4 *>(tiles + j);
        rank += (t.x > mine || (t.x == mine && j < b)) + (t.y > mine || (t.y == mine && j + 1 < b)) +
                (t.z > mine || (t.z == mine && j + 2 < b)) + (t.w > mine || (t.w == mine && j + 3 < b));
    }
    p.order[rank] = b;
}

// ---------------------------------------------------------------------------
// The cut wave's pieces joined: one CTA per (unit, row tile, 16 columns), a
// thread per row; piece weights 2^(m_i - M).
// ---------------------------------------------------------------------------
constexpr int kMergeCols = 16;

__global__ void __launch_bounds__(kM)
prefill_tc_merge_kernel(const __grid_constant__ PrefillParams p, int row_tiles, int ctas) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int r = blockIdx.x, rt = blockIdx.y, c0 = blockIdx.z * kMergeCols, row = threadIdx.x;
    // one round trip for the layout, one for the pieces: every load that may be needed at once
    const int *d = p.tail_info + kTailUnits + r * 8;
    const int tail = p.tail_info[0], q0 = d[0], ntok = d[1], kvh = d[2], h0 = d[3], nh = d[4], first = d[5], last = d[6];
    // (first == last: taken whole and written by its CTA; the bounds hold unless a wait of the kernel before ran out)
    if (r >= tail || first >= last || first < 0 || last >= ctas) return;
    const int row_tokens = p.tile_tokens / row_tiles;
    const int t = row / p.heads_per_tile, h = row - t * p.heads_per_tile, tok = rt * row_tokens + t;
    if (t >= row_tokens || tok >= ntok || h >= nh || q0 < 0 || q0 + tok >= p.num_tokens || kvh < 0 ||
        kvh >= p.num_kv_heads || h0 < 0 || h0 + h >= p.group)
        return;
    float M = kLowestScore, l = 0.f, o[kMergeCols];
#pragma unroll
    for (int e = 0; e < kMergeCols; ++e) o[e] = 0.f;
    for (int c = first; c <= last; c += 2) {   // two pieces at a time, folded into a running maximum
        float m[2], s[2], x[2][kMergeCols];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            m[k] = kLowestScore;
            s[k] = 0.f;
            if (c + k > last) continue;
            const int64_t piece = static_cast<int64_t>(c + k + r) * row_tiles + rt;
            m[k] = p.part_max[piece * kM + row];
            s[k] = p.part_sum[piece * kM + row];
            const float *src = p.part_out + (piece * p.head_dim + c0) * kM + row;
#pragma unroll
            for (int e = 0; e < kMergeCols; ++e) x[k][e] = src[e * kM];
        }
        const float Mn = fmaxf(M, fmaxf(m[0], m[1])), a = fast_exp2(M - Mn), w0 = fast_exp2(m[0] - Mn),
                    w1 = c + 1 <= last ? fast_exp2(m[1] - Mn) : 0.f;
        M = Mn;
        l = l * a + s[0] * w0 + s[1] * w1;
#pragma unroll
        for (int e = 0; e < kMergeCols; ++e) {
            o[e] = fmaf(x[0][e], w0, o[e] * a);
            if (c + 1 <= last) o[e] = fmaf(x[1][e], w1, o[e]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : l;
    const int64_t at = (static_cast<int64_t>(q0 + tok) * p.num_heads + kvh * p.group + h0 + h) * p.head_dim + c0;
#pragma unroll
    for (int e = 0; e < kMergeCols; e += 2) store_pair_as(p.out, p.out_type, at + e, o[e] * inv, o[e + 1] * inv);
}

template <int D, bool kTwoTiles, bool kF16, bool kWide>
cudaError_t launch_impl(const PrefillParams &p, const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tq,
                        int ctas, cudaStream_t stream) {
    auto kern = prefill_tc_kernel<D, kTwoTiles, kF16, kWide>;
    constexpr size_t smem = smem_bytes<D, kTwoTiles>();
    static unsigned long long done = 0;
    cudaError_t e = ensure_smem_limit(kern, smem, done);
    if (e != cudaSuccess) return e;
    if (p.order) {
        const int threads = (p.num_seqs + 31) / 32 * 32;
        if ((e = launch_kernel(prefill_order_kernel, dim3(1), dim3(threads), 0, stream, 1u, p)) != cudaSuccess) return e;
    } else if (p.counter) {
        if ((e = cudaMemsetAsync(p.counter, 0, sizeof(int), stream)) != cudaSuccess) return e;
    }
    if ((e = launch_kernel(kern, dim3(ctas), dim3(kThreads), smem, stream, 1u, tk, tv, tq, p)) != cudaSuccess) return e;
    if (p.nsplit <= 1) return cudaSuccess;
    const int row_tiles = kTwoTiles ? 2 : 1;
    return launch_kernel(prefill_tc_merge_kernel, dim3(p.max_tail, row_tiles, D / kMergeCols), dim3(kM), 0, stream, 1u, p,
                         row_tiles, ctas);
}

template <int D, bool kTwoTiles, bool kWide>
cudaError_t launch_type(const PrefillParams &p, bool f16, const CUtensorMap &tk, const CUtensorMap &tv,
                        const CUtensorMap &tq, int ctas, cudaStream_t stream) {
    return f16 ? launch_impl<D, kTwoTiles, true, kWide>(p, tk, tv, tq, ctas, stream)
               : launch_impl<D, kTwoTiles, false, kWide>(p, tk, tv, tq, ctas, stream);
}

}  // namespace

bool prefill_tc_supported(int head_dim, int block_size, bool contiguous) {
    return (head_dim == 64 || head_dim == 128) &&
           (contiguous || (block_size >= 8 && block_size <= 256 && (block_size & (block_size - 1)) == 0));
}
int prefill_tc_rows() { return kM; }
int prefill_tc_tile() { return kTile; }
int prefill_tc_max_ctas() { return kMaxTail; }
int prefill_tc_box_tokens(int block_size, bool contiguous) { return contiguous || block_size > 64 ? 64 : block_size; }
int prefill_tc_v_box_halves(int head_dim, int block_size, bool contiguous) {
    return prefill_tc_box_tokens(block_size, contiguous) >= 32 ? 1 : head_dim / 64;
}
size_t prefill_tc_info_bytes() { return kTailInts * sizeof(int); }

cudaError_t launch_prefill_tc(const PrefillParams &p, bool two_tiles, bool f16, const CUtensorMap &tk,
                              const CUtensorMap &tv, const CUtensorMap &tq, int ctas, cudaStream_t stream) {
    if (p.head_dim == 64)   // one half: either layout is the wide one
        return two_tiles ? launch_type<64, true, true>(p, f16, tk, tv, tq, ctas, stream)
                         : launch_type<64, false, true>(p, f16, tk, tv, tq, ctas, stream);
    if (prefill_tc_v_box_halves(p.head_dim, p.block_size, p.contig_stride > 0) == 1)
        return two_tiles ? launch_type<128, true, true>(p, f16, tk, tv, tq, ctas, stream)
                         : launch_type<128, false, true>(p, f16, tk, tv, tq, ctas, stream);
    return two_tiles ? launch_type<128, true, false>(p, f16, tk, tv, tq, ctas, stream)
                     : launch_type<128, false, false>(p, f16, tk, tv, tq, ctas, stream);
}

}  // namespace pa
