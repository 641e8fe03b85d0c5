// Rotary positions: heads rotated by their token's position, alone (pa_rope)
// or on the way into the paged cache (pa_rope_and_cache).
//
// Mathematics. Pair i of a head's first rotary_dim dims, (a, b), becomes
//   (a cos t - b sin t, b cos t + a sin t) * factor,  t = position * inv_freq[i];
// the pair is dims (i, i + rotary_dim / 2) in the half layout and (2i, 2i + 1)
// in the interleaved one; dims past rotary_dim pass through. The transpose
// (sin negated) is the gradient of the rotation.
//
// Angles. inv_freq is given in 64 bits. It is turned into a 64-bit fixed-point
// fraction of a full turn (2^64 = one turn), multiplied by the position in
// integers modulo 2^64 -- the reduction modulo a turn costs nothing and is
// exact -- and only the reduced angle is rounded to fp32, as half turns, for
// sincospif. The error is 2^-65 of a turn a position plus one fp32 rounding,
// whatever the position; an fp32 product position * inv_freq would be off by
// 0.004 rad at position 65,536 already. No 64-bit floating point runs.
//
// Bound: HBM (every element read and written once; a rotation is 6 flops a
// pair). So: 16-byte vectors; a thread takes the two vectors that hold its
// pairs (in the half layout the partner of dim i is rotary_dim / 2 further on,
// so no thread needs another's data), and all loads of kUnroll items are in
// flight before the first is used; the angles of a CTA's tokens are computed
// once, into shared memory, and serve every head. Queries, keys and values of
// a token are one list of heads, so the append is one launch. Few tokens: one
// CTA takes fewer heads of a token, so that a step's latency is one item's.
#include <cmath>

#include "device_common.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 128;   // a CTA's threads, unless one head takes more
constexpr int kUnroll = 3;          // items a thread loads before using any
constexpr int kMaxTokensPerCta = 8;

template <typename T>
struct RopeElem;
template <>
struct RopeElem<float> {
    __device__ static float get(float x) { return x; }
    __device__ static float put(float x) { return x; }
};
template <>
struct RopeElem<__nv_bfloat16> {
    __device__ static float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    __device__ static __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }   // one rounding, at the end
};
template <>
struct RopeElem<__half> {
    __device__ static float get(__half x) { return __half2float(x); }
    __device__ static __half put(float x) { return __float2half_rn(x); }
};

// V elements moved at once.
template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
    T e[V];
};

// position * inv_freq as half turns in [-1, 1) (angle / pi).
__device__ __forceinline__ float half_turns(double inv_freq, int position) {
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(inv_freq));
    const int ef = static_cast<int>(bits >> 52) & 0x7ff;
    if (ef == 0x7ff) return __int_as_float(0x7fffffff);   // inf or NaN: NaN
    const uint64_t frac = bits & ((1ull << 52) - 1);
    const uint64_t m = ef ? frac | (1ull << 52) : frac;
    const int e = (ef ? ef : 1) - 1023;
    // |inv_freq| = m * 2^(e - 52); a turn is 2 pi, so turns * 2^64 = m * K * 2^(e - 54)
    // with K = 2^64 * 2 / pi, rounded
    constexpr uint64_t K = 0xA2F9836E4E44152Aull;
    const uint64_t hi = __umul64hi(m, K), lo = m * K;
    const int s = 54 - e;
    uint64_t turn = 0;
    if (s >= 128) turn = 0;
    else if (s >= 64) turn = hi >> (s - 64);
    else if (s > 0) turn = (hi << (64 - s)) | (lo >> s);
    else if (s > -64) turn = lo << -s;
    uint64_t phase = turn * static_cast<uint64_t>(static_cast<int64_t>(position));
    if (bits >> 63) phase = 0 - phase;
    return __ll2float_rn(static_cast<int64_t>(phase)) * 0x1p-63f;
}

template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRopeMaxHeadDim)
rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float2 cs[];   // [tokens of the CTA][rotary_dim / 2]: factor * (cos, sin)
    __shared__ int s_pos[kMaxTokensPerCta];
    __shared__ int64_t s_slot[kMaxTokensPerCta];
    grid_dependency_wait();
    grid_dependents_launch();
    const int pairs = p.rotary_dim / 2;
    const int tok0 = blockIdx.x * p.tokens_per_cta;
    const int ntok = min(p.tokens_per_cta, p.num_tokens - tok0);
    const int nrot = pairs / V;                                  // threads of a head that rotate (two vectors each)
    const int per_head = nrot + (p.head_dim - p.rotary_dim) / V;   // and those that move a vector past rotary_dim
    const int slots = static_cast<int>(blockDim.x) / per_head;   // heads in flight
    const int u = threadIdx.x % per_head, hslot = threadIdx.x / per_head;
    const int head0 = blockIdx.y * p.heads_per_cta;
    const int nheads = min(p.heads_per_cta, p.num_heads + 2 * p.num_kv_heads - head0);
    const int iters = (nheads + slots - 1) / slots;              // per token
    const bool rotates = u < nrot;
    // element offsets of the thread's vectors within a head
    const int off_a = !rotates ? p.rotary_dim + (u - nrot) * V : (kInterleaved && V == 1) ? 2 * u : u * V;
    const int off_b = (kInterleaved && V == 1) ? 2 * u + 1 : pairs + u * V;

    for (int i = threadIdx.x; i < ntok; i += blockDim.x) {
        s_pos[i] = p.positions[tok0 + i];
        if (p.num_kv_heads) s_slot[i] = p.slot_mapping[tok0 + i];
    }
    for (int i = threadIdx.x; i < ntok * pairs; i += blockDim.x) {
        float sn, cn;
        sincospif(half_turns(p.inv_freq[i % pairs], p.positions[tok0 + i / pairs]), &sn, &cn);
        cs[i] = make_float2(cn * p.factor, p.transpose ? -sn * p.factor : sn * p.factor);
    }
    __syncthreads();
    if (hslot >= slots) return;

    using Vec = RopeVec<T, V>;
    const int total = ntok * iters;
    for (int base = 0; base < total; base += kUnroll) {
        Vec a[kUnroll], b[kUnroll];
        const T *src[kUnroll];
        T *dst[kUnroll];
        bool turn[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int it = base + k;
            const int t = it / iters, h = head0 + (it - t * iters) * slots + hslot;
            src[k] = nullptr;
            dst[k] = nullptr;
            turn[k] = false;
            if (it >= total || h >= head0 + nheads || s_pos[t] < 0) continue;   // a negative position: padding
            const int64_t tok = tok0 + t;
            const int kv = h - p.num_heads;
            if (kv < 0) {
                src[k] = static_cast<const T *>(p.x) + tok * p.x_stride + static_cast<int64_t>(h) * p.head_dim;
                dst[k] = static_cast<T *>(p.out) + tok * p.out_stride + static_cast<int64_t>(h) * p.head_dim;
                turn[k] = rotates;
            } else {
                const int64_t slot = s_slot[t];
                if (slot < 0 || slot >= p.num_slots) continue;
                const bool is_v = kv >= p.num_kv_heads;
                const int64_t head = is_v ? kv - p.num_kv_heads : kv;
                src[k] = static_cast<const T *>(is_v ? p.value : p.key) + tok * (is_v ? p.value_stride : p.key_stride) +
                         head * p.head_dim;
                dst[k] = static_cast<T *>(is_v ? p.v_cache : p.k_cache) + (slot * p.num_kv_heads + head) * p.head_dim;
                turn[k] = rotates && !is_v;
            }
            a[k] = *reinterpret_cast<const Vec *>(src[k] + off_a);
            if (rotates) b[k] = *reinterpret_cast<const Vec *>(src[k] + off_b);
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (!dst[k]) continue;
            if (turn[k]) {
                const float2 *c = cs + ((base + k) / iters) * pairs;
                if constexpr (kInterleaved && V > 1) {   // pairs inside each vector
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float2 ca = c[(u * V + e) / 2], cb = c[(pairs + u * V + e) / 2];
                        const float x0 = RopeElem<T>::get(a[k].e[e]), y0 = RopeElem<T>::get(a[k].e[e + 1]);
                        const float x1 = RopeElem<T>::get(b[k].e[e]), y1 = RopeElem<T>::get(b[k].e[e + 1]);
                        a[k].e[e] = RopeElem<T>::put(x0 * ca.x - y0 * ca.y);
                        a[k].e[e + 1] = RopeElem<T>::put(y0 * ca.x + x0 * ca.y);
                        b[k].e[e] = RopeElem<T>::put(x1 * cb.x - y1 * cb.y);
                        b[k].e[e + 1] = RopeElem<T>::put(y1 * cb.x + x1 * cb.y);
                    }
                } else {                                 // a pair across the two vectors
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float2 cc = c[u * V + e];
                        const float x = RopeElem<T>::get(a[k].e[e]), y = RopeElem<T>::get(b[k].e[e]);
                        a[k].e[e] = RopeElem<T>::put(x * cc.x - y * cc.y);
                        b[k].e[e] = RopeElem<T>::put(y * cc.x + x * cc.y);
                    }
                }
            }
            *reinterpret_cast<Vec *>(dst[k] + off_a) = a[k];
            if (rotates) *reinterpret_cast<Vec *>(dst[k] + off_b) = b[k];
        }
    }
}

template <typename T, int V>
cudaError_t launch_rope_vec(RopeParams &p, int sms, cudaStream_t stream) {
    const int per_head = p.rotary_dim / 2 / V + (p.head_dim - p.rotary_dim) / V;
    const int threads = per_head > kRopeThreads ? per_head : kRopeThreads / per_head * per_head;
    const int slots = threads / per_head;
    const int heads = p.num_heads + 2 * p.num_kv_heads;
    // Many tokens: a CTA takes every head of a few tokens (angles shared by all).
    // Few tokens: one item a thread, the heads of a token over several CTAs.
    const bool few = static_cast<int64_t>(p.num_tokens) * heads < static_cast<int64_t>(sms) * slots * 4;
    p.heads_per_cta = few ? slots : heads;
    int tpc = few ? 1 : p.num_tokens / (sms * 8);
    tpc = tpc < 1 ? 1 : tpc > kMaxTokensPerCta ? kMaxTokensPerCta : tpc;
    p.tokens_per_cta = tpc;
    const dim3 grid(static_cast<unsigned>((p.num_tokens + tpc - 1) / tpc),
                    static_cast<unsigned>((heads + p.heads_per_cta - 1) / p.heads_per_cta));
    const size_t smem = static_cast<size_t>(tpc) * (p.rotary_dim / 2) * sizeof(float2);
    return p.interleaved ? launch_kernel(rope_kernel<T, V, true>, grid, dim3(threads), smem, stream, 1u, p)
                         : launch_kernel(rope_kernel<T, V, false>, grid, dim3(threads), smem, stream, 1u, p);
}

// The widest vector whose elements never straddle a pair's halves, the end of
// the rotated part or an alignment boundary of any operand.
int rope_vector(const RopeParams &p, int elem_bytes) {
    auto fits = [&](int v) {
        const int pairs = p.rotary_dim / 2;
        if (pairs % v || (p.head_dim - p.rotary_dim) % v) return false;
        if (p.head_dim / v > kRopeThreads * 2) return false;
        auto ok = [&](const void *ptr, int64_t stride) {
            return reinterpret_cast<uintptr_t>(ptr) % (static_cast<uintptr_t>(v) * elem_bytes) == 0 && stride % v == 0;
        };
        if (!ok(p.x, p.x_stride) || !ok(p.out, p.out_stride)) return false;
        if (p.num_kv_heads && (!ok(p.key, p.key_stride) || !ok(p.value, p.value_stride))) return false;
        return true;
    };
    for (int v = 16 / elem_bytes; v > 1; v /= 2)
        if (v != 4 || elem_bytes == 4)   // 16-byte vectors, then (16-bit types) pairs
            if (fits(v)) return v;
    return 1;
}

}  // namespace

cudaError_t launch_rope(RopeParams &p, int type, int sms, cudaStream_t stream) {
    const int v = rope_vector(p, type == 0 ? 4 : 2);
    if (type == 0) {
        if (v == 4) return launch_rope_vec<float, 4>(p, sms, stream);
        if (v == 2) return launch_rope_vec<float, 2>(p, sms, stream);
        return launch_rope_vec<float, 1>(p, sms, stream);
    }
    if (type == 1) {
        if (v == 8) return launch_rope_vec<__nv_bfloat16, 8>(p, sms, stream);
        if (v == 2) return launch_rope_vec<__nv_bfloat16, 2>(p, sms, stream);
        return launch_rope_vec<__nv_bfloat16, 1>(p, sms, stream);
    }
    if (v == 8) return launch_rope_vec<__half, 8>(p, sms, stream);
    if (v == 2) return launch_rope_vec<__half, 2>(p, sms, stream);
    return launch_rope_vec<__half, 1>(p, sms, stream);
}

}  // namespace pa
