// Heads normed and rotated in one pass: alone (pa_norm_rope), on the way into
// the paged cache (pa_norm_rope_and_cache), and the gradients
// (pa_norm_rope_backward).
//
// Mathematics. A head x of D dims becomes R(y), y = w * x * r with
// r = 1 / sqrt(mean(x^2) + eps) and R the rotation of rope.cu. With g = R^T dout
// (the rotation is orthogonal up to its factor) and u = x * r:
//   dw = sum over rows of g * u,
//   dx = r * (w g - u * mean(w g u)).
//
// Bound: HBM, as the rotation alone: every element is read and written once (the
// gradients read two and write one). The norm doubles the instructions a byte: bf16
// heads of 128 take 0.70 of the issue slots at 0.68 (8,192 tokens x 32 heads, 29.5 us)
// and 0.81 (append of 16,500 x 48, 74.4 us) of the copy rate. So: a row is held by 2^k lanes of one warp, two
// 16-byte vectors a lane (the halves of its pairs), its sum of squares is a butterfly
// of shuffles, and the angles of a CTA's tokens are computed once into shared memory
// while the rows are on their way. Sums and products are fp32; one rounding, at the
// end. The gradient of w is summed in registers over the rows that a thread sees,
// then over the CTA's threads, the CTAs and never by atomics: the same call gives
// the same bits.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "rope_common.cuh"

namespace pa {

namespace {

constexpr int kNormThreads = 128;
constexpr int kNormGradRows = 2;   // rows a thread has in flight, of two operands each
constexpr int kNormGradCtasPerSm = 4;
constexpr int kNormSumThreads = 1024;

// Where a lane's vectors lie within a head: item i of lane l is vector pair
// l + i * lanes of the head's list (pairs that are rotated, then the rest). kFull:
// all of the head is rotated and every lane has one pair of vectors, known at
// compile time, so that no vector of a row hangs on a test (see launch_norm_rows).
template <int V, bool kInterleaved, int kItems, bool kFull>
struct NormLane {
    int off_a[kItems], off_b[kItems], u[kItems];
    bool has_a[kItems], has_b[kItems], turned[kItems];
    __device__ __forceinline__ bool live(int i) const { return kFull || has_a[i]; }
    __device__ __forceinline__ bool two(int i) const { return kFull || has_b[i]; }
    __device__ __forceinline__ bool rotates(int i) const { return kFull || turned[i]; }
    __device__ NormLane(const RopeParams &p, int lane, int lanes) {
        const int pairs = p.rotary_dim / 2;
        const int nrot = pairs / V, pass = (p.head_dim - p.rotary_dim) / V, npass = (pass + 1) / 2;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            u[i] = lane + i * lanes;
            has_a[i] = u[i] < nrot + npass;
            turned[i] = u[i] < nrot;
            has_b[i] = has_a[i] && (turned[i] || u[i] - nrot + npass < pass);
            off_a[i] = !rotates(i) ? p.rotary_dim + (u[i] - nrot) * V : (kInterleaved && V == 1) ? 2 * u[i] : u[i] * V;
            off_b[i] = !rotates(i) ? off_a[i] + npass * V : (kInterleaved && V == 1) ? 2 * u[i] + 1 : pairs + u[i] * V;
        }
    }
};

template <typename T, int V>
__device__ __forceinline__ void unpack(const RopeVec<T, V> &v, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = v.get(0);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 x = v.get2(i);
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ void pack(RopeVec<T, V> &v, const float (&f)[V]) {
    if constexpr (V == 1) {
        v.put(0, f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v.put2(i, make_float2(f[2 * i], f[2 * i + 1]));
    }
}

// The lane's pairs turned by c (cos, sin of its token, [rotary_dim / 2]).
template <int V, bool kInterleaved>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float2 *c, int u, int pairs) {
    if constexpr (V == 1) {
        const float2 t = c[u];
        const float x = a[0], y = b[0];
        a[0] = x * t.x - y * t.y;
        b[0] = y * t.x + x * t.y;
    } else if constexpr (!kInterleaved) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {   // two angles a read
            const float4 t = *reinterpret_cast<const float4 *>(c + u * V + i);
            const float x0 = a[i], y0 = b[i], x1 = a[i + 1], y1 = b[i + 1];
            a[i] = x0 * t.x - y0 * t.y;
            b[i] = y0 * t.x + x0 * t.y;
            a[i + 1] = x1 * t.z - y1 * t.w;
            b[i + 1] = y1 * t.z + x1 * t.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 ta = c[u * (V / 2) + i], tb = c[pairs / 2 + u * (V / 2) + i];
            const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
            a[2 * i] = x * ta.x - y * ta.y;
            a[2 * i + 1] = y * ta.x + x * ta.y;
            b[2 * i] = z * tb.x - w * tb.y;
            b[2 * i + 1] = w * tb.x + z * tb.y;
        }
    }
}

// Sum over the 2^k lanes that hold a row (every lane of the warp takes part).
__device__ __forceinline__ float row_sum(float x, int lanes) {
    for (int d = lanes / 2; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// (cos, sin) * factor of ntok tokens from tok0 on; the transpose negates sin.
__device__ __forceinline__ void fill_angles(const RopeParams &p, float2 *cs, int tok0, int ntok, bool transpose) {
    const int pairs = p.rotary_dim / 2;
    for (int i = threadIdx.x; i < ntok * pairs; i += blockDim.x) {
        const int t = i / pairs;
        float sn, cn;
        sincospif(half_turns(p.inv_freq[i - t * pairs], p.positions[tok0 + t]), &sn, &cn);
        cs[i] = make_float2(cn * p.factor, transpose ? -sn * p.factor : sn * p.factor);
    }
}

// One CTA: tokens_per_cta tokens x heads_per_cta heads of the token's list
// (query heads, key heads, value heads), kRows rows a lane group.
template <typename T, int V, bool kInterleaved, int kItems, int kRows, bool kFull>
__global__ void __launch_bounds__(kNormThreads)
norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    extern __shared__ __align__(16) float2 cs[];
    grid_dependency_wait();
    grid_dependents_launch();
    using Vec = RopeVec<T, V>;
    const int lanes = p.lanes, pairs = p.rotary_dim / 2;
    const int slots = static_cast<int>(blockDim.x) / lanes;
    const int hslot = threadIdx.x / lanes;
    const NormLane<V, kInterleaved, kItems, kFull> at_lane(p, threadIdx.x & (lanes - 1), lanes);
    const int tok0 = blockIdx.x * p.tokens_per_cta;
    const int ntok = min(p.tokens_per_cta, p.num_tokens - tok0);
    const int head0 = blockIdx.y * p.heads_per_cta;
    const int nheads = min(p.heads_per_cta, p.num_heads + 2 * p.num_kv_heads - head0);

    Vec a[kRows][kItems], b[kRows][kItems];
    int tok[kRows], head[kRows];   // token within the CTA (-1: none), head of the list
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int n = hslot + k * slots;
        const int t = n / nheads;
        tok[k] = t < ntok ? t : -1;
        head[k] = head0 + (n - t * nheads);
        if (t >= ntok) continue;
        const int64_t at = tok0 + t;
        const int kv = head[k] - p.num_heads;
        const T *src = kv < 0 ? static_cast<const T *>(p.x) + at * p.x_stride + static_cast<int64_t>(head[k]) * p.head_dim
                       : kv < p.num_kv_heads
                           ? static_cast<const T *>(p.key) + at * p.key_stride + static_cast<int64_t>(kv) * p.head_dim
                           : static_cast<const T *>(p.value) + at * p.value_stride +
                                 static_cast<int64_t>(kv - p.num_kv_heads) * p.head_dim;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (at_lane.live(i)) a[k][i] = *reinterpret_cast<const Vec *>(src + at_lane.off_a[i]);
            if (at_lane.two(i)) b[k][i] = *reinterpret_cast<const Vec *>(src + at_lane.off_b[i]);
        }
    }
    fill_angles(p, cs, tok0, ntok, false);
    __syncthreads();

    const float inv_dim = 1.f / static_cast<float>(p.head_dim);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int kv = head[k] - p.num_heads;
        const bool normed = tok[k] >= 0 && kv < p.num_kv_heads;
        float sum = 0.f;
        if (normed) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                float f[V];
                if (at_lane.live(i)) {
                    unpack<T, V>(a[k][i], f);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum += f[e] * f[e];
                }
                if (at_lane.two(i)) {
                    unpack<T, V>(b[k][i], f);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum += f[e] * f[e];
                }
            }
        }
        sum = row_sum(sum, lanes);
        if (tok[k] < 0) continue;
        const int64_t at = tok0 + tok[k];
        if (p.positions[at] < 0) continue;   // padding
        T *dst;
        if (kv < 0) {
            dst = static_cast<T *>(p.out) + at * p.out_stride + static_cast<int64_t>(head[k]) * p.head_dim;
        } else {
            const int64_t slot = p.slot_mapping[at];
            if (slot < 0 || slot >= p.num_slots) continue;
            dst = kv < p.num_kv_heads
                      ? static_cast<T *>(p.k_cache) + (slot * p.num_kv_heads + kv) * p.head_dim
                      : static_cast<T *>(p.v_cache) + (slot * p.num_kv_heads + kv - p.num_kv_heads) * p.head_dim;
        }
        const T *w = static_cast<const T *>(kv < 0 ? p.weight : p.key_weight);
        const float r = rsqrtf(sum * inv_dim + p.eps);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (normed && at_lane.live(i)) {
                float x[V], y[V], f[V];
                unpack<T, V>(a[k][i], x);
                unpack<T, V>(*reinterpret_cast<const Vec *>(w + at_lane.off_a[i]), f);
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] *= r * f[e];
                if (at_lane.two(i)) {
                    unpack<T, V>(b[k][i], y);
                    unpack<T, V>(*reinterpret_cast<const Vec *>(w + at_lane.off_b[i]), f);
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] *= r * f[e];
                }
                if (at_lane.rotates(i)) turn<V, kInterleaved>(x, y, cs + tok[k] * pairs, at_lane.u[i], pairs);
                pack<T, V>(a[k][i], x);
                if (at_lane.two(i)) pack<T, V>(b[k][i], y);
            }
            if (at_lane.live(i)) *reinterpret_cast<Vec *>(dst + at_lane.off_a[i]) = a[k][i];
            if (at_lane.two(i)) *reinterpret_cast<Vec *>(dst + at_lane.off_b[i]) = b[k][i];
        }
    }
}

// The gradients. The CTAs go round the row groups (tokens_per_cta tokens x
// heads_per_cta heads), so that each leaves one partial sum of w's gradient.
// Measured (bf16, 8,192 tokens x 32 heads of 128): 54.3 us with the sum over the CTAs,
// 0.55 of the copy rate; bound by issue and registers (128 a thread, 16 warps an SM,
// 53 % of the issue slots). One row a lane group in place of two: 62 .. 69 us at 4 ..
// 6 CTAs an SM; two rows and 5 CTAs 57; rows through a ring of cp.async copies 61.
template <typename T, int V, bool kInterleaved, int kItems, int kRows, bool kFull>
__global__ void __launch_bounds__(kNormThreads)
norm_rope_grad_kernel(const __grid_constant__ NormRopeParams p) {
    extern __shared__ __align__(16) float2 cs[];   // two buffers of angles; at the end, the threads' sums
    grid_dependency_wait();
    grid_dependents_launch();
    using Vec = RopeVec<T, V>;
    const int lanes = p.lanes, pairs = p.rotary_dim / 2;
    const int slots = static_cast<int>(blockDim.x) / lanes;
    const int hslot = threadIdx.x / lanes;
    const NormLane<V, kInterleaved, kItems, kFull> at_lane(p, threadIdx.x & (lanes - 1), lanes);
    const int hgroups = (p.num_heads + p.heads_per_cta - 1) / p.heads_per_cta;
    const int tgroups = (p.num_tokens - 1) / p.tokens_per_cta + 1;
    const int groups = tgroups * hgroups;   // (groups write 256 bytes and more on average: no memory holds 2^31)
    const float inv_dim = 1.f / static_cast<float>(p.head_dim);
    const T *w = static_cast<const T *>(p.weight);

    float da[kItems][V], db[kItems][V];
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) da[i][e] = db[i][e] = 0.f;

    int buffer = 0;
    for (int group = blockIdx.x; group < groups; group += static_cast<int>(gridDim.x), buffer ^= 1) {
        const int tgroup = group / hgroups, tok0 = tgroup * p.tokens_per_cta;
        const int head0 = (group - tgroup * hgroups) * p.heads_per_cta;
        const int ntok = min(p.tokens_per_cta, p.num_tokens - tok0);
        const int nheads = min(p.heads_per_cta, p.num_heads - head0);
        float2 *c = cs + buffer * p.tokens_per_cta * pairs;
        Vec a[kRows][kItems], b[kRows][kItems], ga[kRows][kItems], gb[kRows][kItems];
        int tok[kRows], head[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int n = hslot + k * slots;
            const int t = n / nheads;
            head[k] = head0 + (n - t * nheads);
            tok[k] = t < ntok ? t : -1;
            if (t >= ntok) continue;
            const int64_t at = tok0 + t;
            const T *x = static_cast<const T *>(p.x) + at * p.x_stride + static_cast<int64_t>(head[k]) * p.head_dim;
            const T *g = static_cast<const T *>(p.grad_out) + at * p.grad_out_stride + static_cast<int64_t>(head[k]) * p.head_dim;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                if (at_lane.live(i)) {
                    a[k][i] = *reinterpret_cast<const Vec *>(x + at_lane.off_a[i]);
                    ga[k][i] = *reinterpret_cast<const Vec *>(g + at_lane.off_a[i]);
                }
                if (at_lane.two(i)) {
                    b[k][i] = *reinterpret_cast<const Vec *>(x + at_lane.off_b[i]);
                    gb[k][i] = *reinterpret_cast<const Vec *>(g + at_lane.off_b[i]);
                }
            }
        }
        // (the other buffer may still be read; this one's readers passed the barrier of the round between)
        fill_angles(p, c, tok0, ntok, true);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const bool live_row = tok[k] >= 0 && p.positions[tok0 + tok[k]] >= 0;   // (padding has no gradient)
            float sum = 0.f, dot = 0.f;   // of x^2; of w g x
            float x[kItems][2][V], g[kItems][2][V];
            if (live_row) {
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    if (!at_lane.live(i)) continue;
                    float f[V];
                    unpack<T, V>(a[k][i], x[i][0]);
                    unpack<T, V>(ga[k][i], g[i][0]);
                    if (at_lane.two(i)) {
                        unpack<T, V>(b[k][i], x[i][1]);
                        unpack<T, V>(gb[k][i], g[i][1]);
                    }
                    if (at_lane.rotates(i)) turn<V, kInterleaved>(g[i][0], g[i][1], c + tok[k] * pairs, at_lane.u[i], pairs);
                    unpack<T, V>(*reinterpret_cast<const Vec *>(w + at_lane.off_a[i]), f);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        sum += x[i][0][e] * x[i][0][e];
                        dot += f[e] * g[i][0][e] * x[i][0][e];
                    }
                    if (at_lane.two(i)) {
                        unpack<T, V>(*reinterpret_cast<const Vec *>(w + at_lane.off_b[i]), f);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            sum += x[i][1][e] * x[i][1][e];
                            dot += f[e] * g[i][1][e] * x[i][1][e];
                        }
                    }
                }
            }
            sum = row_sum(sum, lanes);
            dot = row_sum(dot, lanes);
            if (!live_row) continue;
            const float r = rsqrtf(sum * inv_dim + p.eps);
            const float mean = dot * r * inv_dim;   // of w g u
            T *dst = static_cast<T *>(p.out) + static_cast<int64_t>(tok0 + tok[k]) * p.out_stride +
                     static_cast<int64_t>(head[k]) * p.head_dim;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                if (!at_lane.live(i)) continue;
                float f[V], y[V];
                Vec v;
                unpack<T, V>(*reinterpret_cast<const Vec *>(w + at_lane.off_a[i]), f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float u = x[i][0][e] * r;
                    da[i][e] += g[i][0][e] * u;
                    y[e] = r * (f[e] * g[i][0][e] - u * mean);
                }
                pack<T, V>(v, y);
                *reinterpret_cast<Vec *>(dst + at_lane.off_a[i]) = v;
                if (!at_lane.two(i)) continue;
                unpack<T, V>(*reinterpret_cast<const Vec *>(w + at_lane.off_b[i]), f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float u = x[i][1][e] * r;
                    db[i][e] += g[i][1][e] * u;
                    y[e] = r * (f[e] * g[i][1][e] - u * mean);
                }
                pack<T, V>(v, y);
                *reinterpret_cast<Vec *>(dst + at_lane.off_b[i]) = v;
            }
        }
    }
    // the CTA's sum of w's gradient, lane group after lane group
    __syncthreads();
    float *sums = reinterpret_cast<float *>(cs);   // [slots][head_dim]
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (at_lane.live(i)) sums[hslot * p.head_dim + at_lane.off_a[i] + e] = da[i][e];
            if (at_lane.two(i)) sums[hslot * p.head_dim + at_lane.off_b[i] + e] = db[i][e];
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.head_dim; d += blockDim.x) {
        float total = 0.f;
        for (int s = 0; s < slots; ++s) total += sums[s * p.head_dim + d];
        p.partials[static_cast<int64_t>(blockIdx.x) * p.head_dim + d] = total;
    }
}

// w's gradient from the CTAs' sums: 8 columns a CTA, 128 threads a column, whose
// loads are all on their way at once.
constexpr int kSumColumns = 8, kSumRows = kNormSumThreads / kSumColumns;
__global__ void __launch_bounds__(kNormSumThreads)
norm_rope_sum_kernel(float *grad_weight, const float *partials, int rows, int head_dim) {
    __shared__ float part[kNormSumThreads / 32][kSumColumns];
    grid_dependency_wait();
    grid_dependents_launch();
    const int col = blockIdx.x * kSumColumns + threadIdx.x % kSumColumns, first = threadIdx.x / kSumColumns;
    float total = 0.f;
    if (col < head_dim) {
#pragma unroll 8
        for (int r = first; r < rows; r += kSumRows) total += partials[static_cast<int64_t>(r) * head_dim + col];
    }
#pragma unroll
    for (int d = kSumColumns; d < 32; d *= 2) total += __shfl_xor_sync(0xffffffffu, total, d);
    if ((threadIdx.x & 31) < kSumColumns) part[threadIdx.x >> 5][threadIdx.x & 31] = total;
    __syncthreads();
    if (threadIdx.x < kSumColumns && col < head_dim) {
        total = 0.f;
#pragma unroll
        for (int s = 0; s < kNormSumThreads / 32; ++s) total += part[s][threadIdx.x];
        grad_weight[col] = total;
    }
}

// Lanes a row: the power of two that holds its vector pairs, a warp at most.
int row_lanes(const RopeParams &p, int v, int *items) {
    const int per_head = p.rotary_dim / 2 / v + ((p.head_dim - p.rotary_dim) / v + 1) / 2;
    int lanes = 1;
    while (lanes < per_head && lanes < 32) lanes *= 2;
    *items = (per_head + lanes - 1) / lanes;
    return lanes;
}

cudaError_t launch_sum(const NormRopeParams &p, int ctas, cudaStream_t stream) {
    return launch_kernel(norm_rope_sum_kernel, dim3((p.head_dim + kSumColumns - 1) / kSumColumns), dim3(kNormSumThreads), 0, stream, 1u,
                         p.grad_weight, p.partials, ctas, p.head_dim);
}

// A head whose dims are all rotated and fill its lanes (the common 64 and 128), by
// the kernel without tests of its vectors: bf16 heads of 128, 8,192 tokens x 32 heads
// 29.5 us (31.9 with the tests), 16,500 tokens x 48 heads of an append 74.4 (79.4).
bool full_head(const RopeParams &p, int v, int lanes) { return p.rotary_dim == p.head_dim && p.head_dim / 2 == v * lanes; }

template <typename T, int V, int kItems, int kRows>
cudaError_t launch_norm_rows(NormRopeParams &p, int rows, cudaStream_t stream) {
    const int heads = p.num_heads + 2 * p.num_kv_heads;
    p.heads_per_cta = std::min(heads, rows);
    p.tokens_per_cta = rows / p.heads_per_cta;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.num_tokens) + p.tokens_per_cta - 1) / p.tokens_per_cta),
                    static_cast<unsigned>((heads + p.heads_per_cta - 1) / p.heads_per_cta));
    const size_t smem = static_cast<size_t>(p.tokens_per_cta) * (p.rotary_dim / 2) * sizeof(float2);
    if constexpr (V > 1 && kItems == 1) {
        if (full_head(p, V, p.lanes))
            return p.interleaved ? launch_kernel(norm_rope_kernel<T, V, true, 1, kRows, true>, grid, dim3(kNormThreads), smem, stream, 1u, p)
                                 : launch_kernel(norm_rope_kernel<T, V, false, 1, kRows, true>, grid, dim3(kNormThreads), smem, stream, 1u, p);
    }
    return p.interleaved ? launch_kernel(norm_rope_kernel<T, V, true, kItems, kRows, false>, grid, dim3(kNormThreads), smem, stream, 1u, p)
                         : launch_kernel(norm_rope_kernel<T, V, false, kItems, kRows, false>, grid, dim3(kNormThreads), smem, stream, 1u, p);
}

template <typename T, int V, int kItems>
cudaError_t launch_norm_items(NormRopeParams &p, int sms, cudaStream_t stream) {
    const int slots = kNormThreads / p.lanes, heads = p.num_heads + 2 * p.num_kv_heads;
    // few rows: one a lane group, so that a step's latency is one row's
    if (kItems > 1 || static_cast<int64_t>(p.num_tokens) * heads <= static_cast<int64_t>(sms) * slots * 2)
        return launch_norm_rows<T, V, kItems, 1>(p, slots, stream);
    // else two or three, whichever leaves fewer of a CTA's lane groups without a row:
    // of 16 lane groups (bf16 heads of 128), 8,192 tokens x 32 heads take two (29.5 us;
    // three 31.5), 16,500 tokens x 48 heads three (74.4 us; two 86.7)
    auto used = [&](int rows) {   // rows a CTA has, of those it could have, in 1/1024
        const int per = std::min(heads, rows), groups = (heads + per - 1) / per;
        return static_cast<int64_t>(rows / per) * heads * 1024 / (static_cast<int64_t>(rows) * groups);
    };
    return used(3 * slots) > used(2 * slots) ? launch_norm_rows<T, V, kItems, kItems == 1 ? 3 : 1>(p, 3 * slots, stream)
                                             : launch_norm_rows<T, V, kItems, kItems == 1 ? 2 : 1>(p, 2 * slots, stream);
}

template <typename T, int V, int kItems>
cudaError_t launch_grad_items(NormRopeParams &p, int sms, cudaStream_t stream) {
    constexpr int kRows = kItems == 1 ? kNormGradRows : 1;
    const int slots = kNormThreads / p.lanes;
    const bool few = static_cast<int64_t>(p.num_tokens) * p.num_heads <= static_cast<int64_t>(sms) * slots * 2;
    const int rows = few ? slots : slots * kRows;
    p.heads_per_cta = std::min(p.num_heads, rows);
    p.tokens_per_cta = rows / p.heads_per_cta;
    const int64_t groups = ((static_cast<int64_t>(p.num_tokens) + p.tokens_per_cta - 1) / p.tokens_per_cta) *
                           ((p.num_heads + p.heads_per_cta - 1) / p.heads_per_cta);
    const int ctas = static_cast<int>(std::min<int64_t>(groups, static_cast<int64_t>(sms) * kNormGradCtasPerSm));
    const size_t smem = std::max(static_cast<size_t>(2) * p.tokens_per_cta * (p.rotary_dim / 2) * sizeof(float2),
                                 static_cast<size_t>(slots) * p.head_dim * sizeof(float));
    auto kern = p.interleaved ? norm_rope_grad_kernel<T, V, true, kItems, kRows, false> : norm_rope_grad_kernel<T, V, false, kItems, kRows, false>;
    if constexpr (V > 1 && kItems == 1) {
        if (full_head(p, V, p.lanes))
            kern = p.interleaved ? norm_rope_grad_kernel<T, V, true, 1, kRows, true> : norm_rope_grad_kernel<T, V, false, 1, kRows, true>;
    }
    const cudaError_t e = launch_kernel(kern, dim3(ctas), dim3(kNormThreads), smem, stream, 1u, p);
    return e != cudaSuccess ? e : launch_sum(p, ctas, stream);
}

template <typename T, int V>
cudaError_t launch_norm_vec(NormRopeParams &p, int sms, cudaStream_t stream) {
    int items;
    p.lanes = row_lanes(p, V, &items);
    if constexpr (V * sizeof(T) < 16) {   // (a head is 256 dims at most: 32 lanes of two 16-byte vectors hold it)
        if (items > 1)
            return p.grad_out ? launch_grad_items<T, V, 4>(p, sms, stream) : launch_norm_items<T, V, 4>(p, sms, stream);
    }
    return p.grad_out ? launch_grad_items<T, V, 1>(p, sms, stream) : launch_norm_items<T, V, 1>(p, sms, stream);
}

// The widest vector whose elements never straddle a pair's halves, the end of
// the rotated part or an alignment boundary of any operand.
int norm_vector(const NormRopeParams &p, int elem_bytes) {
    auto fits = [&](int v) {
        if ((p.rotary_dim / 2) % v || (p.head_dim - p.rotary_dim) % v) return false;
        auto ok = [&](const void *ptr, int64_t stride) {
            return reinterpret_cast<uintptr_t>(ptr) % (static_cast<uintptr_t>(v) * elem_bytes) == 0 && stride % v == 0;
        };
        if (!ok(p.x, p.x_stride) || !ok(p.out, p.out_stride) || !ok(p.weight, 0)) return false;
        if (p.grad_out && !ok(p.grad_out, p.grad_out_stride)) return false;
        return !p.num_kv_heads || (ok(p.key, p.key_stride) && ok(p.value, p.value_stride) && ok(p.key_weight, 0));
    };
    for (int v = 16 / elem_bytes; v > 1; v /= 2)
        if (v != 4 || elem_bytes == 4)   // 16-byte vectors, then pairs
            if (fits(v)) return v;
    return 1;
}

}  // namespace

// The partial sums of the gradients' CTAs.
size_t norm_rope_grad_workspace(int head_dim, int sms) {
    return static_cast<size_t>(sms) * kNormGradCtasPerSm * head_dim * sizeof(float);
}

cudaError_t launch_norm_rope(NormRopeParams &p, int type, int sms, cudaStream_t stream) {
    if (p.num_tokens == 0) return launch_sum(p, 0, stream);   // (the gradients alone come here with none)
    const int v = norm_vector(p, type == 0 ? 4 : 2);
    if (type == 0) {
        if (v == 4) return launch_norm_vec<float, 4>(p, sms, stream);
        if (v == 2) return launch_norm_vec<float, 2>(p, sms, stream);
        return launch_norm_vec<float, 1>(p, sms, stream);
    }
    if (type == 1) {
        if (v == 8) return launch_norm_vec<__nv_bfloat16, 8>(p, sms, stream);
        if (v == 2) return launch_norm_vec<__nv_bfloat16, 2>(p, sms, stream);
        return launch_norm_vec<__nv_bfloat16, 1>(p, sms, stream);
    }
    if (v == 8) return launch_norm_vec<__half, 8>(p, sms, stream);
    if (v == 2) return launch_norm_vec<__half, 2>(p, sms, stream);
    return launch_norm_vec<__half, 1>(p, sms, stream);
}

}  // namespace pa
