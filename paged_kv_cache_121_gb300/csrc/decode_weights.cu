// One decode step that also adds the weight it gave every cached token to a table:
// out = softmax(scale q K^T) V, weights = decay * weights + sum over the query heads
// of each KV head of their softmax weights.
//
// Mathematics. A token's weight needs its row's maximum and sum, which stand only
// after the last token. So the scores are kept (4 bytes a token and query head: 3 %
// of the K and V bytes of a group of 4 heads of 128) and turned into weights by the
// CTA that made them, once the row's statistics are merged; no second pass over K.
//
// Bound: HBM, K and V read once for every 16 query heads of a KV head. How:
//  * One cluster of up to 8 CTAs = one sequence x a group of KV heads; each CTA takes
//    a range of the context. A warp owns one KV head and every sets-th tile of the
//    range and fetches its own tiles by 16-byte asynchronous copies into a ring of
//    its own (24 KB), through the block table, token by token: any block size will do
//    and no warp waits for another before the end. Rows are swizzled (16-byte chunk ^
//    token & 7), so that the matrix loads have no bank conflicts.
//  * 16-bit caches: products on mma.m16n8k16 (M = the query heads, 16 at most a pass;
//    bound by memory, so the wider tcgen05 tiles would stand empty), softmax online in
//    base 2. fp32: CUDA cores.
//  * The weights of V enter the products in parts of the caches' type: three of bf16, which
//    hold fp32's 24 bits (two left 2^-17 of a weight, seen in fp32 outputs), or two of fp16,
//    22 bits and none below 2^-32 of a row's largest weight. Errors of fp32 outputs against
//    64 bits, relative in norm, at 300 .. 32,768 tokens: 1.6e-7 .. 6.3e-7, half of what the
//    same in fp32 operations leaves.
//  * The warps' states meet in shared memory, the cluster's CTAs through distributed
//    shared memory; each CTA merges a slice of the outputs and, for itself, every
//    row's maximum and sum, and then goes through its own scores (in L2 still).
//    One launch, no atomics: the same call gives the same bits.
//  * More than 16 query heads a KV head: the passes follow one another in the CTA, each with
//    its own reads of K and V (64 heads on one, 16 x 32,768 tokens: 539 us).
//
// Measured (16 sequences of 4,164 tokens, 32 / 8 heads of 128, bf16, blocks of 16):
// 58.1 us, 0.72 of the copy rate (the decode alone, whose copies TMA makes, takes 44).
// It reads 4.8 TB/s from its start to its end, the merge and the weights at the end
// included; 54.4 us with bf16 weights in two parts and V's products summed on the tensor
// cores over the whole context. Block ids looked at as soon as they were loaded, and the scores turned
// into weights one token a thread: 67.9 us.
#include <algorithm>

#include "async_copy.cuh"
#include "internal.h"
#include "mma_tile.cuh"
#include "packed_math.cuh"
#include "weights_common.cuh"

namespace pa {

namespace {

constexpr int kRingBytes = 24 * 1024;   // a warp's tiles in flight

template <typename T, int D>
struct StepCfg {
    static constexpr bool kFloat = sizeof(T) == 4;
    static constexpr int kTile = kFloat ? 8 : 16;                  // tokens
    static constexpr int kRow = D * static_cast<int>(sizeof(T));   // bytes of one head's row
    static constexpr int kChunks = kRow / 16;
    static constexpr int kStage = 2 * kTile * kRow;                // K, then V
    static constexpr int kStages = kRingBytes / kStage;
    static constexpr int kStateStride = D + 8;                     // floats a row: 8-byte stores of 4 rows in 32 banks
    static constexpr int kState = 32 + kRowsPerTile * kStateStride;
    static_assert(kState * 4 <= kRingBytes, "a warp's state takes its ring's place");
};

// Weights as a sum of 16-bit parts, two weights a register: bf16 takes the upper halves of what is left, whose 24 bits
// three parts hold exactly.
template <bool kF16, int kParts>
__device__ __forceinline__ void split_parts(float x, float y, uint32_t (&part)[kParts]) {
    if constexpr (kF16) {
        split_f16x2(x, y, part[0], part[1]);
    } else {
#pragma unroll
        for (int n = 0; n < kParts; ++n) {
            const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
            part[n] = __byte_perm(a, b, 0x7632);
            x -= __uint_as_float(a & 0xffff0000u);
            y -= __uint_as_float(b & 0xffff0000u);
        }
    }
}

// One warp's query rows and running state, 16-bit caches.
template <typename T, int D>
struct StepTile {
    using C = StepCfg<T, D>;
    static constexpr bool kF16 = std::is_same<T, __half>::value;
    static constexpr int kParts = kF16 ? 2 : 3;   // of a weight
    // fp16 weights are raised by 2^7, as far as the slack below leaves room: what its smallest numbers cut off lies
    // that much lower.
    static constexpr float kRaise = kF16 ? 7.f : 0.f;
    WarpState<D> st;
    uint32_t qa[D / 16][4];

    __device__ __forceinline__ void start(const T *query, float *, int rows, int lane) {   // query: the warp's first row
        st.init();
        const uint32_t *q0 = reinterpret_cast<const uint32_t *>(query) + (lane >> 2) * (D / 2);
        load_query_fragments<D>(qa, q0, q0 + 8 * (D / 2), (lane >> 2) < rows, (lane >> 2) + 8 < rows, lane);
    }

    // One tile of `valid` tokens; scores: the first row's, at the tile's first token.
    __device__ __forceinline__ void add(const unsigned char *stage, const float *, float *scores, int64_t score_stride,
                                        int rows, int valid, float scale, int lane) {
        const int r = lane >> 2, q4 = lane & 3;
        const uint32_t kbase = smem_addr(stage), vbase = kbase + C::kTile * C::kRow;
        float s[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float odd[4] = {0.f, 0.f, 0.f, 0.f};
            s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
            const int tok = 8 * j + (lane & 7);
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 2) {
                const int c = 2 * kk + (lane >> 3);
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4(kbase + tok * C::kRow + ((c ^ (tok & 7)) << 4), b0, b1, b2, b3);
                mma_16816<kF16>(s[j], qa[kk], b0, b1);
                mma_16816<kF16>(odd, qa[kk + 1], b2, b3);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = (s[j][e] + odd[e]) * scale;
        }
        if (valid < C::kTile) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (8 * j + 2 * q4 + e >= valid) s[j][e] = s[j][2 + e] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {   // (the rows of scores are padded to whole tiles)
            float *to = scores + r * score_stride + 8 * j + 2 * q4;
            if (r < rows) *reinterpret_cast<float2 *>(to) = make_float2(s[j][0], s[j][1]);
            if (r + 8 < rows) *reinterpret_cast<float2 *>(to + 8 * score_stride) = make_float2(s[j][2], s[j][3]);
        }
        float m0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float m1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
        for (int d = 1; d < 4; d *= 2) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
        }
        // The reference (a maximum less kRaise) moves only where a score passes that maximum by kRescaleSlack. (Differences:
        // a sum with a score of 2^27 would round by 8, and a weight leave fp16.)
        const bool up0 = m0 - st.m0 > kRescaleSlack + kRaise, up1 = m1 - st.m1 > kRescaleSlack + kRaise;
        if (__any_sync(0xffffffffu, up0 || up1)) {
            const float n0 = up0 ? m0 - kRaise : st.m0, n1 = up1 ? m1 - kRaise : st.m1;
            const float a0 = up0 ? fast_exp2(st.m0 - n0) : 1.f, a1 = up1 ? fast_exp2(st.m1 - n1) : 1.f;
            st.m0 = n0;
            st.m1 = n1;
            st.l0 *= a0;
            st.l1 *= a1;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                st.o[i][0] *= a0;
                st.o[i][1] *= a0;
                st.o[i][2] *= a1;
                st.o[i][3] *= a1;
            }
        }
        // (a row that has seen nothing but -inf has m = -inf: its weights are zeros)
        const float b0 = st.m0 == -INFINITY ? 0.f : st.m0, b1 = st.m1 == -INFINITY ? 0.f : st.m1;
        uint32_t part[kParts][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float p0 = fast_exp2(s[j][0] - b0), p1 = fast_exp2(s[j][1] - b0);
            const float p2 = fast_exp2(s[j][2] - b1), p3 = fast_exp2(s[j][3] - b1);
            st.l0 += p0 + p1;
            st.l1 += p2 + p3;
            uint32_t of0[kParts], of1[kParts];
            split_parts<kF16>(p0, p1, of0);
            split_parts<kF16>(p2, p3, of1);
#pragma unroll
            for (int n = 0; n < kParts; ++n) {
                part[n][2 * j] = of0[n];
                part[n][2 * j + 1] = of1[n];
            }
        }
        // A tile's products are summed from zero, then added: the tensor cores cut off what reaches below a sum's last bit,
        // always in one direction, which over the tiles of a context came to 2^-17 of an output.
#pragma unroll
        for (int dn = 0; dn < D / 8; dn += 2) {
            const int mi = lane >> 3;
            const int tok = (mi & 1) * 8 + (lane & 7), c = dn + (mi >> 1);
            uint32_t v[4];
            ldmatrix_x4_trans(vbase + tok * C::kRow + ((c ^ (tok & 7)) << 4), v[0], v[1], v[2], v[3]);
            float o[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int n = kParts - 1; n >= 0; --n) {   // the smallest first
                mma_16816<kF16>(o[0], part[n], v[0], v[1]);
                mma_16816<kF16>(o[1], part[n], v[2], v[3]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    float *to = st.o[dn + i];
                    unpair(add2(pair(to[e], to[e + 1]), pair(o[i][e], o[i][e + 1])), to[e], to[e + 1]);
                }
        }
    }

    // State rows: (max, sum) of each of 16 rows, then the rows' sums of V.
    __device__ __forceinline__ void leave(float *state, int, int lane) {
        const int r = lane >> 2, q4 = lane & 3;
        st.reduce_sums();
#pragma unroll
        for (int dn = 0; dn < D / 8; ++dn) {
            float *o = state + 32 + r * C::kStateStride + 8 * dn + 2 * q4;
            *reinterpret_cast<float2 *>(o) = make_float2(st.o[dn][0], st.o[dn][1]);
            *reinterpret_cast<float2 *>(o + 8 * C::kStateStride) = make_float2(st.o[dn][2], st.o[dn][3]);
        }
        if (q4 == 0) {
            *reinterpret_cast<float2 *>(state + 2 * r) = make_float2(st.m0, st.l0);
            *reinterpret_cast<float2 *>(state + 2 * (r + 8)) = make_float2(st.m1, st.l1);
        }
    }
};

// fp32 caches: lane = (token of 8, quarter of the dims) for the scores, D / 32 dims a lane for the sums of V.
template <int D>
struct StepTile<float, D> {
    using C = StepCfg<float, D>;
    static constexpr int kDims = D / 32;
    float m[kRowsPerTile], l[kRowsPerTile], o[kRowsPerTile][kDims];

    __device__ __forceinline__ void start(const float *query, float *q, int rows, int lane) {
#pragma unroll
        for (int r = 0; r < kRowsPerTile; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int d = 0; d < kDims; ++d) o[r][d] = 0.f;
        }
        for (int i = lane; i < rows * D; i += 32) q[i] = query[i];
        __syncwarp();
    }

    __device__ __forceinline__ void add(const unsigned char *stage, const float *q, float *scores, int64_t score_stride,
                                        int rows, int valid, float scale, int lane) {
        const int tok = lane >> 2, quarter = lane & 3;
        const unsigned char *k = stage + tok * C::kRow;
        const unsigned char *v = stage + C::kTile * C::kRow;
#pragma unroll
        for (int r = 0; r < kRowsPerTile; ++r) {
            if (r >= rows) break;
            float s = 0.f;
#pragma unroll 4
            for (int c = quarter; c < C::kChunks; c += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(k + ((c ^ (tok & 7)) << 4));
                const float4 b = *reinterpret_cast<const float4 *>(q + r * D + 4 * c);
                s += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            s = tok < valid ? s * scale : -INFINITY;
            if (quarter == 0) scores[r * score_stride + tok] = s;
            float top = s;
#pragma unroll
            for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (top > m[r]) {
                const float a = fast_exp2(m[r] - top);
                m[r] = top;
                l[r] *= a;
#pragma unroll
                for (int d = 0; d < kDims; ++d) o[r][d] *= a;
            }
            const float p = fast_exp2(s - (m[r] == -INFINITY ? 0.f : m[r]));
            if (quarter == 0) l[r] += p;
#pragma unroll
            for (int t = 0; t < C::kTile; ++t) {
                const float pt = __shfl_sync(0xffffffffu, p, 4 * t);
#pragma unroll
                for (int d = 0; d < kDims; ++d) {   // dim lane + 32 d of token t
                    const int dim = lane + 32 * d;
                    const float x = *reinterpret_cast<const float *>(v + t * C::kRow + (((dim >> 2) ^ (t & 7)) << 4) + (dim & 3) * 4);
                    o[r][d] += pt * x;
                }
            }
        }
    }

    __device__ __forceinline__ void leave(float *state, int rows, int lane) {
#pragma unroll
        for (int r = 0; r < kRowsPerTile; ++r) {
            if (r >= rows) break;
            float sum = l[r];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
            for (int d = 0; d < kDims; ++d) state[32 + r * C::kStateStride + lane + 32 * d] = o[r][d];
            if (lane == 0) *reinterpret_cast<float2 *>(state + 2 * r) = make_float2(m[r], sum);
        }
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(256, 1)
decode_weights_kernel(const __grid_constant__ DecodeWeightsParams p) {
    using C = StepCfg<T, D>;
    extern __shared__ __align__(128) unsigned char smem[];   // the warps' rings, later their states; fp32: query rows
    __shared__ float2 s_row[8][kRowsPerTile];                // a KV head's rows: maximum, 1 / sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nwarps = blockDim.x >> 5;
    grid_dependency_wait();

    const int b = blockIdx.z, head0 = blockIdx.y * p.heads_per_cta;
    const int sets_log = __ffs(p.sets) - 1;   // (a power of two)
    const int head = head0 + (warp >> sets_log), set = warp & (p.sets - 1);   // this warp's KV head, its share of the tiles
    const int given = p.context_lens[b];
    int len = max(0, min(given, p.max_ctx));
    len = static_cast<int>(min(static_cast<int64_t>(len), static_cast<int64_t>(p.max_blocks) * p.block_size));
    const int tok_begin = min(len, static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * p.part_tokens, static_cast<int64_t>(len))));
    const int tok_end = static_cast<int>(min(static_cast<int64_t>(len), static_cast<int64_t>(tok_begin) + p.part_tokens));
    const int all_tiles = (tok_end - tok_begin + C::kTile - 1) / C::kTile;
    const int tiles = all_tiles > set ? (all_tiles - set + p.sets - 1) / p.sets : 0;   // this warp's
    const int32_t *table = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
    unsigned char *ring = smem + warp * kRingBytes;
    const uint32_t ring_addr = smem_addr(ring);
    float *q_rows = reinterpret_cast<float *>(smem + nwarps * kRingBytes) + warp * (C::kFloat ? kRowsPerTile * D : 0);
    const int64_t token_bytes = static_cast<int64_t>(p.num_kv_heads) * C::kRow;
    const unsigned char *k_head = static_cast<const unsigned char *>(p.k_cache) + head * C::kRow;
    const unsigned char *v_head = static_cast<const unsigned char *>(p.v_cache) + head * C::kRow;

    auto first_token = [&](int i) { return tok_begin + (set + i * p.sets) * C::kTile; };
    // Block and place in it of the lane's token of tile i (place -1: nothing to read). The block is only loaded here
    // and looked at a tile later: waited for at once it cost 700 cycles a tile.
    auto look_up = [&](int i, int &blk, int &in) {
        const int t = first_token(i) + lane;
        in = -1;
        if (i >= tiles || lane >= C::kTile || t >= tok_end) return;
        const int j = t / p.block_size;
        in = t - j * p.block_size;
        blk = table[j];
    };
    auto fetch = [&](int i, int blk, int in) {
        if (i < tiles) {
            const bool in_pool = in >= 0 && static_cast<unsigned>(blk) < static_cast<unsigned>(p.num_blocks);
            const int64_t slot = in_pool ? static_cast<int64_t>(blk) * p.block_size + in : -1;
            // A lane copies chunk c of every kStep-th token. The slots are read ahead: a copy is ordered behind the
            // shuffles before it.
            constexpr int kCopies = C::kTile * C::kChunks / 32, kStep = 32 / C::kChunks;
            const int r0 = lane / C::kChunks, c = lane % C::kChunks;
            int64_t from[kCopies];
#pragma unroll
            for (int n = 0; n < kCopies; ++n) from[n] = __shfl_sync(0xffffffffu, slot, r0 + n * kStep);
            const uint32_t k_dst = ring_addr + (i % C::kStages) * C::kStage, v_dst = k_dst + C::kTile * C::kRow;
            const bool all = __all_sync(0xffffffffu, slot >= 0 || lane >= C::kTile);
#pragma unroll
            for (int n = 0; n < kCopies; ++n) {
                const int t = r0 + n * kStep;
                const uint32_t to = t * C::kRow + ((c ^ (t & 7)) << 4);
                const int64_t off = from[n] * token_bytes + c * 16;
                if (all) {
                    copy16(k_dst + to, k_head + off);
                    copy16(v_dst + to, v_head + off);
                } else {
                    copy16_or_zeros(k_dst + to, k_head + (from[n] < 0 ? 0 : off), from[n] >= 0);
                    copy16_or_zeros(v_dst + to, v_head + (from[n] < 0 ? 0 : off), from[n] >= 0);
                }
            }
        }
        copy_commit();
    };

    // the old weights are on their way to L2 while the tiles are
    if (p.decay != 0.f)
        for (int j = 0; j < p.heads_per_cta; ++j) {
            const float *w = p.weights + (static_cast<int64_t>(b) * p.num_kv_heads + head0 + j) * p.weights_stride;
            for (int t = tok_begin + 32 * static_cast<int>(threadIdx.x); t < tok_end; t += 32 * blockDim.x)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(w + t));
        }

    for (int first = 0; first < p.group; first += kRowsPerTile) {   // 16 query heads of each KV head a pass
        const int rows = min(kRowsPerTile, p.group - first);
        const int64_t row0 = static_cast<int64_t>(b) * p.num_heads + head * p.group + first;   // the warp's first row
        StepTile<T, D> tile;
        tile.start(static_cast<const T *>(p.query) + row0 * D, q_rows, rows, lane);
        int blk[2] = {0, 0}, in[2];   // tiles looked up, not fetched: the next one and the one behind it
        look_up(0, blk[0], in[0]);
        look_up(1, blk[1], in[1]);
        auto fetch_next = [&](int i) {
            fetch(i, blk[0], in[0]);
            blk[0] = blk[1];
            in[0] = in[1];
            look_up(i + 2, blk[1], in[1]);
        };
        for (int i = 0; i < C::kStages - 1; ++i) fetch_next(i);
        float *scores = p.scores + row0 * p.score_stride;
        for (int i = 0; i < tiles; ++i) {
            fetch_next(i + C::kStages - 1);
            copy_wait<C::kStages - 1>();
            __syncwarp();
            const int t0 = first_token(i);
            tile.add(ring + (i % C::kStages) * C::kStage, q_rows, scores + t0, p.score_stride, rows, min(C::kTile, tok_end - t0),
                     p.scale_log2, lane);
            __syncwarp();   // the stage is free
        }
        copy_wait<0>();
        if (first + kRowsPerTile >= p.group) grid_dependents_launch();
        __syncwarp();
        float *state = reinterpret_cast<float *>(ring);
        tile.leave(state, rows, lane);
        cluster_sync_all();   // every state of the cluster can be read

        const int nsplit = p.nsplit, states = nsplit * p.sets;
        const uint32_t base = smem_addr(smem);
        auto state_addr = [&](int j, int n) {   // state n of the cluster's CTAs and warps for KV head j of the group
            return cluster_map(base + static_cast<uint32_t>((j * p.sets + (n & (p.sets - 1))) * kRingBytes), n >> sets_log);
        };
        // Every row's statistics, and a slice of the outputs: 4 dims of one row a thread. The states are read eight at a
        // time, all on their way before the first is used.
        auto merge = [&](int j, int r, int d, float4 &acc) {   // (maximum, sum) of a row; d >= 0: its dims d .. d + 3 too
            float top = -INFINITY, sum = 0.f;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int n0 = 0; n0 < states; n0 += 8) {
                float2 ml[8];
                float4 o[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    ml[n] = make_float2(-INFINITY, 0.f);
                    o[n] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (n0 + n < states) {
                        const uint32_t at = state_addr(j, n0 + n);
                        ml[n] = ld_cluster_f32x2(at + 8 * r);
                        if (d >= 0) o[n] = ld_cluster_f32x4(at + 4 * (32 + r * C::kStateStride + d));
                    }
                }
                float up = top;
#pragma unroll
                for (int n = 0; n < 8; ++n) up = fmaxf(up, ml[n].x);
                const float ref = up == -INFINITY ? 0.f : up, fade = fast_exp2(top - ref);
                sum *= fade;
                acc.x *= fade;
                acc.y *= fade;
                acc.z *= fade;
                acc.w *= fade;
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float f = fast_exp2(ml[n].x - ref);   // (an empty state's is zero)
                    sum += f * ml[n].y;
                    acc.x += f * o[n].x;
                    acc.y += f * o[n].y;
                    acc.z += f * o[n].z;
                    acc.w += f * o[n].w;
                }
                top = up;
            }
            return make_float2(top, sum);
        };
        const int rank = static_cast<int>(cluster_rank());
        const int total = p.heads_per_cta * rows * (D / 4);
        const int slice = (total + nsplit - 1) / nsplit;
        for (int i = rank * slice + threadIdx.x; i < min(total, (rank + 1) * slice); i += blockDim.x) {
            const int j = i / (rows * (D / 4)), rem = i - j * rows * (D / 4);
            const int r = rem / (D / 4), d = 4 * (rem - r * (D / 4));
            float4 acc;
            const float2 ml = merge(j, r, d, acc);
            const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
            const int64_t at = (static_cast<int64_t>(b) * p.num_heads + (head0 + j) * p.group + first + r) * D + d;
            store_pair_as(p.out, p.out_type, at, acc.x * inv, acc.y * inv);
            store_pair_as(p.out, p.out_type, at + 2, acc.z * inv, acc.w * inv);
        }
        for (int i = threadIdx.x; i < p.heads_per_cta * rows; i += blockDim.x) {
            const int j = i / rows, r = i - j * rows;
            float4 acc;
            const float2 ml = merge(j, r, -1, acc);
            // (a row that weighs nothing: zeros; NaN stays)
            s_row[j][r] = make_float2(ml.y == 0.f || ml.x == -INFINITY ? 0.f : ml.x, ml.y == 0.f ? 0.f : 1.f / ml.y);
        }
        __syncthreads();
        // This CTA's scores become weights, four tokens a thread and kItems of those at once: every load of a round is on
        // its way before the first is used.
        constexpr int kItems = 4;
        const int quads = (tok_end - tok_begin + 3) / 4, items = p.heads_per_cta * quads;
        const int64_t scores0 = (static_cast<int64_t>(b) * p.num_heads + head0 * p.group + first) * p.score_stride + tok_begin;
        float *const weights0 = p.weights + (static_cast<int64_t>(b) * p.num_kv_heads + head0) * p.weights_stride + tok_begin;
        for (int i0 = threadIdx.x; i0 < items; i0 += blockDim.x * kItems) {
            int head_of[kItems], at[kItems];   // KV head of the group (-1: none), first token
            float w[kItems][4], old[kItems][4];
#pragma unroll
            for (int n = 0; n < kItems; ++n) {
                const int i = i0 + n * blockDim.x, j = i / quads;
                head_of[n] = i < items ? j : -1;
                at[n] = 4 * (i - j * quads);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[n][e] = 0.f;
                    // the newest token's weight starts in the first pass
                    const int t = tok_begin + at[n] + e;
                    const bool read = i < items && t < tok_end && (first > 0 || (t != given - 1 && p.decay != 0.f));
                    old[n][e] = read ? weights0[j * p.weights_stride + at[n] + e] : 0.f;
                }
            }
            for (int r0 = 0; r0 < rows; r0 += 4) {
                float4 s[kItems][4];
#pragma unroll
                for (int n = 0; n < kItems; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (head_of[n] >= 0 && r0 + r < rows)
                            s[n][r] = *reinterpret_cast<const float4 *>(
                                p.scores + scores0 + (static_cast<int64_t>(head_of[n]) * p.group + r0 + r) * p.score_stride + at[n]);
#pragma unroll
                for (int n = 0; n < kItems; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (head_of[n] >= 0 && r0 + r < rows) {
                            const float2 ml = s_row[head_of[n]][r0 + r];
                            w[n][0] += fast_exp2(s[n][r].x - ml.x) * ml.y;
                            w[n][1] += fast_exp2(s[n][r].y - ml.x) * ml.y;
                            w[n][2] += fast_exp2(s[n][r].z - ml.x) * ml.y;
                            w[n][3] += fast_exp2(s[n][r].w - ml.x) * ml.y;
                        }
            }
#pragma unroll
            for (int n = 0; n < kItems; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (head_of[n] >= 0 && tok_begin + at[n] + e < tok_end)
                        weights0[head_of[n] * p.weights_stride + at[n] + e] = w[n][e] + (first > 0 ? old[n][e] : p.decay * old[n][e]);
        }
        cluster_sync_all();   // the peers have read this CTA's states
    }
}

// KV heads a CTA serves, its warps, the CTAs of a context. Two CTAs of 4 warps an SM, or, where even
// single heads and clusters of 8 leave SMs without one, one of 8 warps.
struct StepPlan {
    int heads, warps, nsplit, part_tokens;
};

StepPlan plan_step(int num_seqs, int num_kv_heads, int max_ctx, int sms) {
    StepPlan pl;
    const int64_t slots = 2 * static_cast<int64_t>(sms);
    pl.heads = 4;
    while (pl.heads > 1 && (num_kv_heads % pl.heads != 0 ||
                            static_cast<int64_t>(num_seqs) * (num_kv_heads / pl.heads) * kMaxClusterSplits * 4 < slots * 3))
        pl.heads /= 2;
    const int64_t units = static_cast<int64_t>(num_seqs) * (num_kv_heads / pl.heads);
    pl.warps = units * kMaxClusterSplits <= sms ? 8 : 4;
    // a CTA's warps have two tiles each at least
    const int64_t most = std::max(1, max_ctx / (pl.warps / pl.heads * 32));
    pl.nsplit = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kMaxClusterSplits, slots / units, most})));
    const int64_t part = (static_cast<int64_t>(max_ctx) + pl.nsplit - 1) / pl.nsplit;
    pl.part_tokens = static_cast<int>(std::min<int64_t>((part + 15) / 16 * 16, INT32_MAX / 16 * 16));
    return pl;
}

template <typename T, int D>
cudaError_t launch_step(DecodeWeightsParams &p, const StepPlan &pl, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(pl.warps) * (kRingBytes + (sizeof(T) == 4 ? kRowsPerTile * D * 4 : 0));
    const dim3 grid(static_cast<unsigned>(pl.nsplit), static_cast<unsigned>(p.num_kv_heads / pl.heads),
                    static_cast<unsigned>(p.num_seqs));
    auto kern = decode_weights_kernel<T, D>;
    static unsigned long long done = 0;
    const cudaError_t e = ensure_smem_limit(kern, 8 * kRingBytes + (sizeof(T) == 4 ? 8 * 1024 : 0), done);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, grid, dim3(32 * pl.warps), smem, stream, static_cast<unsigned>(pl.nsplit), p);
}

}  // namespace

int64_t decode_weights_score_stride(int max_ctx) { return (static_cast<int64_t>(max_ctx) + 15) / 16 * 16; }

cudaError_t launch_decode_weights(DecodeWeightsParams &p, int type, int head_dim, int sms, cudaStream_t stream) {
    StepPlan pl = plan_step(p.num_seqs, p.num_kv_heads, p.max_ctx, sms);
    if (type == 0) pl.warps = 4;   // (fp32 query rows take the room of the other four)
    p.heads_per_cta = pl.heads;
    p.sets = pl.warps / pl.heads;
    p.nsplit = pl.nsplit;
    p.part_tokens = pl.part_tokens;
    if (head_dim == 128)
        return type == 0   ? launch_step<float, 128>(p, pl, stream)
               : type == 1 ? launch_step<__nv_bfloat16, 128>(p, pl, stream)
                           : launch_step<__half, 128>(p, pl, stream);
    return type == 0   ? launch_step<float, 64>(p, pl, stream)
           : type == 1 ? launch_step<__nv_bfloat16, 64>(p, pl, stream)
                       : launch_step<__half, 64>(p, pl, stream);
}

}  // namespace pa
