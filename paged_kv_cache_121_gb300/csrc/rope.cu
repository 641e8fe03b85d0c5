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
// sincospif. The fraction is rounded to nearest, so the angle is off by at most
// 2^-65 of a turn a position (plus 2^-72 a position and radian of inv_freq, from
// the constant 2 / pi) and one fp32 rounding; an fp32 product position * inv_freq
// would be off by 0.004 rad at position 65,536 already. No 64-bit floating point runs.
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

#include "internal.h"
#include "rope_common.cuh"

namespace pa {

namespace {

// 128 threads x 3 (token, head) rows a thread, all loaded before any is used.
// Measured on GB300 over 128 .. 320 threads x 2 .. 4 rows (bf16, heads of 128;
// 8,192 tokens x 40 heads / 16,400-token append of 32 + 8 + 8 heads): this one
// 31.0 / 64.8 us, 0.80 / 0.92 of the copy rate; the others 33.0 .. 37.3 / 69.7
// .. 85.8 us. Small CTAs keep some loading while others wait for their angles.
constexpr int kRopeThreads = 128;
constexpr int kUnroll = 3;
static_assert(kRopeMaxHeadDim <= 2 * kRopeThreads, "a head's threads fit a CTA");

// One CTA: tokens_per_cta tokens x heads_per_cta heads of the token's list
// (query heads, key heads, value heads), at most `slots` x kUnroll of them.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float2 cs[];   // [tokens of the CTA][rotary_dim / 2]: factor * (cos, sin)
    grid_dependency_wait();
    grid_dependents_launch();
    const int pairs = p.rotary_dim / 2;
    const int tok0 = blockIdx.x * p.tokens_per_cta;
    const int ntok = min(p.tokens_per_cta, p.num_tokens - tok0);
    const int nrot = pairs / V;                                    // threads of a head that rotate (two vectors each)
    const int pass = (p.head_dim - p.rotary_dim) / V;              // vectors past rotary_dim: two a thread too
    const int npass = (pass + 1) / 2, per_head = nrot + npass;
    const int slots = static_cast<int>(blockDim.x) / per_head;     // heads in flight
    const int hslot = threadIdx.x / per_head, u = threadIdx.x - hslot * per_head;
    const int head0 = blockIdx.y * p.heads_per_cta;
    const int nheads = min(p.heads_per_cta, p.num_heads + 2 * p.num_kv_heads - head0);
    const bool rotates = u < nrot;
    const bool two = rotates || u - nrot + npass < pass;
    // element offsets of the thread's vectors within a head
    const int off_a = !rotates ? p.rotary_dim + (u - nrot) * V : (kInterleaved && V == 1) ? 2 * u : u * V;
    const int off_b = !rotates ? off_a + npass * V : (kInterleaved && V == 1) ? 2 * u + 1 : pairs + u * V;

    // every load of the CTA is on its way before the angles are computed
    using Vec = RopeVec<T, V>;
    Vec a[kUnroll], b[kUnroll];
    int tok[kUnroll], head[kUnroll];   // token within the CTA (-1: none), head of the list
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
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
        a[k] = *reinterpret_cast<const Vec *>(src + off_a);
        if (two) b[k] = *reinterpret_cast<const Vec *>(src + off_b);
    }

    for (int i = threadIdx.x; i < ntok * pairs; i += blockDim.x) {
        const int t = i / pairs;
        float sn, cn;
        sincospif(half_turns(p.inv_freq[i - t * pairs], p.positions[tok0 + t]), &sn, &cn);
        cs[i] = make_float2(cn * p.factor, p.transpose ? -sn * p.factor : sn * p.factor);
    }
    __syncthreads();

#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        if (tok[k] < 0) continue;
        const int64_t at = tok0 + tok[k];
        if (p.positions[at] < 0) continue;   // padding
        const int kv = head[k] - p.num_heads;
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
        if (rotates && kv < p.num_kv_heads) {
            const float2 *c = cs + tok[k] * pairs;
            if constexpr (V == 1) {                  // the pair is the two elements
                const float2 cc = c[u];
                const float x = a[k].get(0), y = b[k].get(0);
                a[k].put(0, x * cc.x - y * cc.y);
                b[k].put(0, y * cc.x + x * cc.y);
            } else if constexpr (kInterleaved) {     // pairs inside each vector
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float2 ca = c[u * (V / 2) + i], cb = c[pairs / 2 + u * (V / 2) + i];
                    const float2 x = a[k].get2(i), y = b[k].get2(i);
                    a[k].put2(i, make_float2(x.x * ca.x - x.y * ca.y, x.y * ca.x + x.x * ca.y));
                    b[k].put2(i, make_float2(y.x * cb.x - y.y * cb.y, y.y * cb.x + y.x * cb.y));
                }
            } else {                                 // pairs across the two vectors
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float2 c0 = c[u * V + 2 * i], c1 = c[u * V + 2 * i + 1];
                    const float2 x = a[k].get2(i), y = b[k].get2(i);
                    a[k].put2(i, make_float2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y));
                    b[k].put2(i, make_float2(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y));
                }
            }
        }
        *reinterpret_cast<Vec *>(dst + off_a) = a[k];
        if (two) *reinterpret_cast<Vec *>(dst + off_b) = b[k];
    }
}

template <typename T, int V>
cudaError_t launch_rope_vec(RopeParams &p, int sms, cudaStream_t stream) {
    const int per_head = p.rotary_dim / 2 / V + ((p.head_dim - p.rotary_dim) / V + 1) / 2;
    const int slots = kRopeThreads / per_head;
    const int threads = slots * per_head;
    const int heads = p.num_heads + 2 * p.num_kv_heads;
    // Few (token, head) rows: one a thread, so that a step's latency is one row's.
    // Many: kUnroll rows a thread, of whole tokens where they fit (angles shared by their heads).
    const bool few = static_cast<int64_t>(p.num_tokens) * heads <= static_cast<int64_t>(sms) * slots * 2;
    const int rows = few ? slots : slots * kUnroll;
    p.heads_per_cta = heads < rows ? heads : rows;
    p.tokens_per_cta = rows / p.heads_per_cta;
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.num_tokens) + p.tokens_per_cta - 1) / p.tokens_per_cta),
                    static_cast<unsigned>((heads + p.heads_per_cta - 1) / p.heads_per_cta));
    const size_t smem = static_cast<size_t>(p.tokens_per_cta) * (p.rotary_dim / 2) * sizeof(float2);
    return p.interleaved ? launch_kernel(rope_kernel<T, V, true>, grid, dim3(threads), smem, stream, 1u, p)
                         : launch_kernel(rope_kernel<T, V, false>, grid, dim3(threads), smem, stream, 1u, p);
}

// The widest vector whose elements never straddle a pair's halves, the end of
// the rotated part or an alignment boundary of any operand.
int rope_vector(const RopeParams &p, int elem_bytes) {
    auto fits = [&](int v) {
        const int pairs = p.rotary_dim / 2;
        if (pairs % v || (p.head_dim - p.rotary_dim) % v) return false;
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
