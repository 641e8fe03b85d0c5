// The weights that several query tokens a sequence gave each cached token, on the
// CUDA cores (fp32 caches; 16-bit caches take prefill_weights_tc.cu).
//
// Mathematics. weights[t] gains the sum over rows i (query tokens that count x query
// heads of the KV head) of 2^((s_it - b_i) scale) / l_i, s = q.k, scale times log2(e), b_i
// the row's score that weighs most, l_i the sum of those powers. The sum over rows needs
// every row's b_i and l_i, so K is passed
// over twice: first the rows' statistics, then the sums. The scores are computed again
// in the second pass: kept they would be 4 bytes a pair to write and read, some
// hundred times the bytes of K.
//
// Bound: fp32 multiply-adds (2 D a pair and pass). One tile product serves both passes:
// a CTA holds 64 rows of one operand and streams 64-row tiles of the other, both
// transposed in shared memory so that a thread's 4 x 4 products read two 16-byte
// vectors a dim. First pass: queries held, keys streamed; second: the other way round,
// so that what is reduced over (keys, then rows) is always the streamed side.
// Measured as the path of 16-bit caches too, before prefill_weights_tc.cu: 8 chunks of
// 200 .. 1,500 tokens behind up to 2,500, 32 / 8 heads of 128, 4.6 ms (28 TFLOP/s).
#include <algorithm>

#include "internal.h"
#include "weights_common.cuh"

namespace pa {

namespace {

constexpr int kSide = 64;            // rows of either operand's tile
constexpr int kThreads = 256;        // 16 x 16, 4 x 4 products each
constexpr int kPitch = kSide + 4;    // floats of one dim's row

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
// Rows i0 .. i0 + 63 of an operand, transposed to [dim][row]; row(i) is null for one that does not exist (zeros).
template <int D, typename Row>
__device__ __forceinline__ void load_tile(float *tile, Row row) {
    constexpr int kVecs = D / 4;
    for (int i = threadIdx.x; i < kSide * kVecs; i += kThreads) {
        const int r = i % kSide, c = i / kSide;
        const float *src = row(r);
        const float4 x = src ? load4(src + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        float *to = tile + 4 * c * kPitch + r;
        to[0] = x.x;
        to[kPitch] = x.y;
        to[2 * kPitch] = x.z;
        to[3 * kPitch] = x.w;
    }
}

// s[i][j] = held row 4 y + i . streamed row 4 x + j
template <int D>
__device__ __forceinline__ void tile_product(const float *held, const float *streamed, float (&s)[4][4]) {
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
    for (int d = 0; d < D; ++d) {
        const float4 a = load4(held + d * kPitch + 4 * y), b = load4(streamed + d * kPitch + 4 * x);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] += av[i] * bv[j];
    }
}

template <int D>
struct Operands {
    const PrefillWeightsParams &p;
    const WeightSeq &s;
    int b, head;
    // row r of the KV head's queries
    __device__ const float *query(int64_t r) const {
        if (r >= static_cast<int64_t>(s.count) * p.group) return nullptr;
        const int64_t token = s.q0 + r / p.group;
        return static_cast<const float *>(p.query) + (token * p.num_heads + head * p.group + r % p.group) * D;
    }
    __device__ const float *key(int t) const {   // (a block outside the pool reads as zeros)
        if (t >= s.ctx) return nullptr;
        const int blk = p.block_tables[static_cast<int64_t>(b) * p.max_blocks + t / p.block_size];
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) return nullptr;
        const int64_t slot = static_cast<int64_t>(blk) * p.block_size + t % p.block_size;
        return static_cast<const float *>(p.k_cache) + (slot * p.num_kv_heads + head) * D;
    }
};

// The rows' statistics: grid (row tiles x pieces of the context, KV heads, sequences).
template <int D>
__global__ void __launch_bounds__(kThreads)
weight_stats_simt_kernel(const __grid_constant__ PrefillWeightsParams p) {
    extern __shared__ __align__(16) float tiles[];
    float *held = tiles, *streamed = tiles + D * kPitch;
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.z, head = blockIdx.y;
    const int piece = blockIdx.x % p.nsplit, tile = blockIdx.x / p.nsplit;
    const WeightSeq s = weight_seq(p, b);
    const int64_t rows = static_cast<int64_t>(s.count) * p.group, r0 = static_cast<int64_t>(tile) * kSide;
    if (r0 >= rows) return;
    const Operands<D> at{p, s, b, head};
    const int last = static_cast<int>(min(rows, r0 + kSide) - 1);
    const int reach = s.sees(last / p.group);   // keys that any row of the tile sees
    const int key_tiles = (reach + kSide - 1) / kSide;
    const int per = (key_tiles + p.nsplit - 1) / p.nsplit;
    load_tile<D>(held, [&](int r) { return at.query(r0 + r); });
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const float sign = p.scale_log2 < 0.f ? -1.f : 1.f, size = fabsf(p.scale_log2);
    int sees[4];
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 4 * y + i;
        sees[i] = r < rows ? s.sees(static_cast<int>(r / p.group)) : 0;
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    for (int kt = piece * per; kt < min(key_tiles, (piece + 1) * per); ++kt) {
        __syncthreads();
        load_tile<D>(streamed, [&](int r) { return at.key(kt * kSide + r); });
        __syncthreads();
        float q[4][4];
        tile_product<D>(held, streamed, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[i][j] = kt * kSide + 4 * x + j < sees[i] ? q[i][j] * sign : -INFINITY;
                top = fmaxf(top, q[i][j]);
            }
            const float base = top == -INFINITY ? 0.f : top;
            l[i] *= fast_exp2((m[i] - base) * size);
            m[i] = top;
#pragma unroll
            for (int j = 0; j < 4; ++j) l[i] += fast_exp2((q[i][j] - base) * size);
        }
    }
    // the 16 threads of a row
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float top = m[i];
#pragma unroll
        for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        float sum = l[i] * fast_exp2((m[i] - (top == -INFINITY ? 0.f : top)) * size);
#pragma unroll
        for (int d = 1; d < 16; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const int64_t r = r0 + 4 * y + i;
        if (x == 0 && r < rows)
            leave_stats(p, piece, s.stat0 + r / p.group, static_cast<int>(head * p.group + r % p.group), top, sum);
    }
}

// The sums over rows: grid (key tiles, KV heads, sequences).
template <int D>
__global__ void __launch_bounds__(kThreads)
weight_sums_simt_kernel(const __grid_constant__ PrefillWeightsParams p) {
    extern __shared__ __align__(16) float tiles[];
    __shared__ float2 stats[kSide];
    __shared__ int sees[kSide];
    float *held = tiles, *streamed = tiles + D * kPitch;
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = blockIdx.z, head = blockIdx.y, t0 = blockIdx.x * kSide;
    const WeightSeq s = weight_seq(p, b);
    if (t0 >= s.ctx) return;
    const Operands<D> at{p, s, b, head};
    const int64_t rows = static_cast<int64_t>(s.count) * p.group;
    // the first token whose queries see the tile's first key
    const int first = max(0, t0 - s.past);
    load_tile<D>(held, [&](int r) { return at.key(t0 + r); });
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t r0 = static_cast<int64_t>(first) * p.group / kSide * kSide; r0 < rows; r0 += kSide) {
        __syncthreads();
        load_tile<D>(streamed, [&](int r) { return at.query(r0 + r); });
        if (threadIdx.x < kSide) {
            const int64_t r = r0 + threadIdx.x;
            const bool live = r < rows;
            stats[threadIdx.x] = live ? p.rows[(s.stat0 + r / p.group) * p.num_heads + head * p.group + r % p.group] : make_float2(0.f, 0.f);
            sees[threadIdx.x] = live ? s.sees(static_cast<int>(r / p.group)) : 0;
        }
        __syncthreads();
        float q[4][4];
        tile_product<D>(held, streamed, q);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 row = stats[4 * x + j];
            const int n = sees[4 * x + j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + 4 * y + i < n) sum[i] += fast_exp2((q[i][j] - row.x) * p.scale_log2) * row.y;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int d = 1; d < 16; d *= 2) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], d);
        const int t = t0 + 4 * y + i;
        if (x == 0 && t < s.ctx) {
            float *w = p.weights + (static_cast<int64_t>(b) * p.num_kv_heads + head) * p.weights_stride + t;
            *w = sum[i] + (t < s.fresh && p.decay != 0.f ? p.decay * *w : 0.f);
        }
    }
}

__global__ void __launch_bounds__(kThreads) weight_merge_kernel(const __grid_constant__ PrefillWeightsParams p) {
    grid_dependency_wait();
    grid_dependents_launch();
    merge_stats(p, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x);
}

template <int D>
cudaError_t launch_simt(const PrefillWeightsParams &p, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(2) * D * kPitch * sizeof(float);
    static unsigned long long stats_done = 0, sums_done = 0;
    cudaError_t e = ensure_smem_limit(weight_stats_simt_kernel<D>, smem, stats_done);
    if (e == cudaSuccess) e = ensure_smem_limit(weight_sums_simt_kernel<D>, smem, sums_done);
    if (e != cudaSuccess) return e;
    const int64_t row_tiles = (static_cast<int64_t>(p.max_count) * p.group + kSide - 1) / kSide;
    const dim3 rows(static_cast<unsigned>(row_tiles * p.nsplit), static_cast<unsigned>(p.num_kv_heads),
                    static_cast<unsigned>(p.num_seqs));
    e = launch_kernel(weight_stats_simt_kernel<D>, rows, dim3(kThreads), smem, stream, 1u, p);
    if (e == cudaSuccess && p.nsplit > 1)
        e = launch_kernel(weight_merge_kernel, dim3(static_cast<unsigned>((p.stat_rows * p.num_heads + kThreads - 1) / kThreads)),
                          dim3(kThreads), 0, stream, 1u, p);
    if (e != cudaSuccess) return e;
    const dim3 keys(static_cast<unsigned>((static_cast<int64_t>(p.max_ctx) + kSide - 1) / kSide),
                    static_cast<unsigned>(p.num_kv_heads), static_cast<unsigned>(p.num_seqs));
    return launch_kernel(weight_sums_simt_kernel<D>, keys, dim3(kThreads), smem, stream, 1u, p);
}

}  // namespace

int prefill_weights_simt_rows() { return kSide; }

cudaError_t launch_prefill_weights_simt(const PrefillWeightsParams &p, int head_dim, cudaStream_t stream) {
    return head_dim == 128 ? launch_simt<128>(p, stream) : launch_simt<64>(p, stream);
}

}  // namespace pa
