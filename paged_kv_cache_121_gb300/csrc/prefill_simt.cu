// Attention of several query tokens a sequence on the CUDA cores: fp32, and
// 16-bit caches whose blocks the tensor-core kernel does not take.
//
// Mathematics: O = softmax(scale Q K^T + mask) V row by row, the softmax held
// as a running maximum m and sum l in base 2 while the keys stream past:
//   m' = max(m, max_j s_j), l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   O' = O 2^(m - m') + sum_j 2^(s_j - m') v_j,    out = O / l  (0 when l = 0).
//
// Layout: a CTA takes 16 RT packed rows (query tokens x the query heads of one
// KV head, so that a K/V tile is read once for all of them) and streams the
// context through shared memory in tiles of 32 tokens, every operand as fp32.
// 256 threads as 16 x 16: a thread holds RT rows x 2 keys of the scores and RT
// rows x D / 16 dims of O in registers; the 16 threads of a row sit in one
// half-warp, so the softmax reductions are shuffles. The next tile is fetched
// while one is computed. Bound: the fp32 pipe and the shared-memory loads that
// feed it; for small batches latency, so RT = 1 where a sequence has at most 16
// rows (a taller tile would multiply rows that are not there) or 64-row tiles
// would not fill the SMs (three prompts of 12 to 47 tokens: 10.3 -> 6.0 us with
// the tile fetched ahead).
// Contexts are cut into pieces (partials through the workspace, merged after)
// when there are fewer tiles than CTA slots.
#include "internal.h"
#include "prompt_common.cuh"

namespace pa {

namespace {

constexpr int kKeys = 32;       // context tokens per tile
constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf16_bits_to_float(v.x & 0xffffu), bf16_bits_to_float(v.x >> 16),
                       bf16_bits_to_float(v.y & 0xffffu), bf16_bits_to_float(v.y >> 16));
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

template <int D, int RT>
struct SimtCfg {
    static constexpr int kRows = 16 * RT;
    static constexpr int kStride = D + 4;       // floats: rows 4 banks apart, 16-byte aligned
    static constexpr int kPStride = kKeys + 4;
    static constexpr size_t kSmem =
        sizeof(float) * (static_cast<size_t>(kRows + 2 * kKeys) * kStride + kRows * kPStride);
};

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreads)
prefill_simt_kernel(const __grid_constant__ PrefillParams p) {
    using C = SimtCfg<D, RT>;
    extern __shared__ __align__(16) float smem_f[];
    float *qs = smem_f, *ks = qs + C::kRows * C::kStride, *vs = ks + kKeys * C::kStride,
          *ps = vs + kKeys * C::kStride;
    __shared__ int found[2];
    grid_dependency_wait();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (tid < 32) {
        int tile = 0;
        const int b = prefill_find_tile(p, blockIdx.x, tid, tile);
        if (tid == 0) {
            found[0] = b;
            found[1] = tile;
        }
    }
    __syncthreads();
    const int b = found[0];
    if (b < 0) return;
    const PrefillSeq s = prefill_seq(p, b);
    const int tok0 = found[1] * p.tile_tokens;                    // first query token of the tile, in the sequence
    const int ntok = min(p.tile_tokens, s.qlen - tok0);
    const int kvh = blockIdx.y / p.ntile, h0 = (blockIdx.y % p.ntile) * p.heads_per_tile;
    const int nh = min(p.heads_per_tile, p.group - h0);
    const int rows = ntok * nh;                                   // row r: token tok0 + r / nh, head h0 + r % nh

    int sees[RT];
    float m[RT], l[RT];
    float4 o[RT][D / 64];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = ty * RT + i;
        sees[i] = r < rows ? prefill_sees(p, s, tok0 + r / nh) : 0;
        m[i] = kLowestScore;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int most = prefill_sees(p, s, tok0 + ntok - 1);         // the last token sees the most
    const int tiles = (most + kKeys - 1) / kKeys;
    const int part = blockIdx.z;
    const int t_begin = static_cast<int>(static_cast<int64_t>(tiles) * part / p.nsplit);
    const int t_end = static_cast<int>(static_cast<int64_t>(tiles) * (part + 1) / p.nsplit);

    const int64_t row_elems = static_cast<int64_t>(p.num_kv_heads) * D;
    const int lr = tid >> 3, lc = (tid & 7) * 4;                  // this thread's row of the tile, first column
    float4 kx[D / 32], vx[D / 32];                                // the next tile's, on its way while one is computed
    auto fetch = [&](int t) {
        const int tok = t * kKeys + lr;
        int64_t at = -1;                                           // row of the cache; -1: not read, zeros
        if (t < t_end && tok < s.ctx) {
            if (p.contig_stride > 0) {
                at = static_cast<int64_t>(b) * p.contig_stride + tok;
            } else {
                const int blk = p.block_tables[static_cast<int64_t>(b) * p.max_blocks + tok / p.block_size];
                if (blk >= 0 && blk < p.num_blocks) at = static_cast<int64_t>(blk) * p.block_size + tok % p.block_size;
            }
        }
        const T *kr = static_cast<const T *>(p.k_cache) + at * row_elems + kvh * D + lc;
        const T *vr = static_cast<const T *>(p.v_cache) + at * row_elems + kvh * D + lc;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            kx[c] = vx[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (at >= 0) {
                kx[c] = load4(kr + c * 32);
                vx[c] = load4(vr + c * 32);
            }
        }
    };
    fetch(t_begin);
    // the rows' queries, scaled to base-2 scores
    for (int i = tid; i < C::kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            const int64_t row = static_cast<int64_t>(s.q0 + tok0 + r / nh) * p.num_heads + kvh * p.group + h0 + r % nh;
            v = load4(static_cast<const T *>(p.query) + row * D + c);
            v.x *= p.scale_log2;
            v.y *= p.scale_log2;
            v.z *= p.scale_log2;
            v.w *= p.scale_log2;
        }
        *reinterpret_cast<float4 *>(qs + r * C::kStride + c) = v;
    }
    for (int t = t_begin; t < t_end; ++t) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            *reinterpret_cast<float4 *>(ks + lr * C::kStride + lc + c * 32) = kx[c];
            *reinterpret_cast<float4 *>(vs + lr * C::kStride + lc + c * 32) = vx[c];
        }
        __syncthreads();
        fetch(t + 1);
        float sc[RT][2];
#pragma unroll
        for (int i = 0; i < RT; ++i) sc[i][0] = sc[i][1] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            const float4 k0 = *reinterpret_cast<const float4 *>(ks + tx * C::kStride + d);
            const float4 k1 = *reinterpret_cast<const float4 *>(ks + (tx + 16) * C::kStride + d);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const float4 q = *reinterpret_cast<const float4 *>(qs + (ty * RT + i) * C::kStride + d);
                sc[i][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, sc[i][0]))));
                sc[i][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, sc[i][1]))));
            }
        }
        const int j0 = t * kKeys + tx;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if (j0 >= sees[i]) sc[i][0] = -INFINITY;
            if (j0 + 16 >= sees[i]) sc[i][1] = -INFINITY;
            float mx = fmaxf(sc[i][0], sc[i][1]);
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m[i], mx);
            const float alpha = exp2f(m[i] - mn);
            m[i] = mn;
            const float p0 = exp2f(sc[i][0] - mn), p1 = exp2f(sc[i][1] - mn);
            l[i] = l[i] * alpha + (p0 + p1);                       // this thread's keys: summed over the 16 at the end
            float *pr = ps + (ty * RT + i) * C::kPStride;
            pr[tx] = p0;
            pr[tx + 16] = p1;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                o[i][c].x *= alpha;
                o[i][c].y *= alpha;
                o[i][c].z *= alpha;
                o[i][c].w *= alpha;
            }
        }
        __syncwarp();
#pragma unroll 4
        for (int j = 0; j < kKeys; ++j) {
            float4 v[D / 64];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) v[c] = *reinterpret_cast<const float4 *>(vs + j * C::kStride + c * 64 + tx * 4);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const float w = ps[(ty * RT + i) * C::kPStride + j];
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    o[i][c].x = fmaf(w, v[c].x, o[i][c].x);
                    o[i][c].y = fmaf(w, v[c].y, o[i][c].y);
                    o[i][c].z = fmaf(w, v[c].z, o[i][c].z);
                    o[i][c].w = fmaf(w, v[c].w, o[i][c].w);
                }
            }
        }
        __syncwarp();
    }
    grid_dependents_launch();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        const int r = ty * RT + i;
        if (r >= rows) continue;
        const float inv = l[i] > 0.f ? 1.f / l[i] : l[i];          // 0: an empty row; NaN stays NaN
        const int64_t row = static_cast<int64_t>(s.q0 + tok0 + r / nh) * p.num_heads + kvh * p.group + h0 + r % nh;
        if (p.nsplit > 1) {
            const int64_t pr = row * p.nsplit + part;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                *reinterpret_cast<float4 *>(p.part_out + pr * D + c * 64 + tx * 4) =
                    make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv, o[i][c].w * inv);
            if (tx == 0) {
                p.part_max[pr] = l[i] == 0.f ? -INFINITY : m[i];
                p.part_sum[pr] = l[i];
            }
        } else {
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int64_t at = row * D + c * 64 + tx * 4;
                store_pair_as(p.out, p.out_type, at, o[i][c].x * inv, o[i][c].y * inv);
                store_pair_as(p.out, p.out_type, at + 2, o[i][c].z * inv, o[i][c].w * inv);
            }
        }
    }
}

// Merge the pieces of every row that belongs to a sequence: one warp a row.
// Weights 2^(m_i - M) l_i of the normalised pieces; rows outside every
// sequence are left as they were.
template <int D>
__global__ void __launch_bounds__(128)
prefill_simt_merge_kernel(const __grid_constant__ PrefillParams p) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= static_cast<int64_t>(p.num_tokens) * p.num_heads) return;
    const int64_t tok = row / p.num_heads;
    if (tok < p.query_start[0] || tok >= p.query_start[p.num_seqs]) return;
    float M = kLowestScore, l = 0.f;
    for (int i = 0; i < p.nsplit; ++i) M = fmaxf(M, p.part_max[row * p.nsplit + i]);
    float o[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
    for (int i = 0; i < p.nsplit; ++i) {
        const float sum = p.part_sum[row * p.nsplit + i];
        if (sum == 0.f) continue;
        const float w = exp2f(p.part_max[row * p.nsplit + i] - M) * sum;
        l += w;
        const float *src = p.part_out + (row * p.nsplit + i) * D + lane * (D / 32);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] = fmaf(w, src[e], o[e]);
    }
    const float inv = l > 0.f ? 1.f / l : l;
#pragma unroll
    for (int e = 0; e < D / 32; e += 2)
        store_pair_as(p.out, p.out_type, row * D + lane * (D / 32) + e, o[e] * inv, o[e + 1] * inv);
}

template <typename T, int D, int RT>
cudaError_t launch_simt(const PrefillParams &p, dim3 grid, cudaStream_t stream) {
    auto kern = prefill_simt_kernel<T, D, RT>;
    static unsigned long long done = 0;
    cudaError_t e = ensure_smem_limit(kern, SimtCfg<D, RT>::kSmem, done);
    if (e != cudaSuccess) return e;
    e = launch_kernel(kern, grid, dim3(kThreads), SimtCfg<D, RT>::kSmem, stream, 1u, p);
    if (e != cudaSuccess || p.nsplit == 1) return e;
    const int64_t rows = static_cast<int64_t>(p.num_tokens) * p.num_heads;
    return launch_kernel(prefill_simt_merge_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream,
                         1u, p);
}

template <typename T>
cudaError_t launch_simt_type(const PrefillParams &p, bool tall, dim3 grid, cudaStream_t stream) {
    if (p.head_dim == 128) return tall ? launch_simt<T, 128, 4>(p, grid, stream) : launch_simt<T, 128, 1>(p, grid, stream);
    if (p.head_dim == 64) return tall ? launch_simt<T, 64, 4>(p, grid, stream) : launch_simt<T, 64, 1>(p, grid, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

int prefill_simt_rows(bool tall) { return tall ? 64 : 16; }

cudaError_t launch_prefill_simt(const PrefillParams &p, int kv_type, bool tall, dim3 grid, cudaStream_t stream) {
    if (kv_type == 0) return launch_simt_type<float>(p, tall, grid, stream);
    if (kv_type == 1) return launch_simt_type<__nv_bfloat16>(p, tall, grid, stream);
    return launch_simt_type<__half>(p, tall, grid, stream);
}

}  // namespace pa
