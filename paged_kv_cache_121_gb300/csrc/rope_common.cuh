// What the rotary kernels share (rope.cu, norm_rope.cu): the vectors they move
// and the angle of a position.
#pragma once

#include "prompt_common.cuh"

namespace pa {

// Heads normed, then rotated (norm_rope.cu): the rotation's arguments, and the
// norm's. With grad_out the gradients: out is then the gradient of x.
struct NormRopeParams : RopeParams {
    const void *weight, *key_weight;   // [head_dim], of x's type
    const void *grad_out;              // [num_tokens, num_heads, head_dim], or null
    int64_t grad_out_stride;
    float *grad_weight;                // [head_dim]
    float *partials;                   // [CTAs][head_dim]
    float eps;
    int lanes;                         // lanes that hold a row (set by the launcher)
};

// V elements moved at once, two at a time in and out of fp32 (the one
// rounding is at the end). 16-bit elements stay packed in 32-bit words until
// they are used: unpacked early they cost the bf16 kernel 20 registers.
template <typename T, int V>
struct alignas(4 * V) RopeVec {      // fp32
    float e[V];
    __device__ float get(int i) const { return e[i]; }
    __device__ void put(int i, float x) { e[i] = x; }
    __device__ float2 get2(int i) const { return make_float2(e[2 * i], e[2 * i + 1]); }
    __device__ void put2(int i, float2 x) {
        e[2 * i] = x.x;
        e[2 * i + 1] = x.y;
    }
};
template <typename T, int V>
struct alignas(2 * V) RopeVec16 {
    uint32_t w[V / 2];
};
template <int V>
struct alignas(2 * V) RopeVec<__nv_bfloat16, V> : RopeVec16<__nv_bfloat16, V> {
    __device__ float2 get2(int i) const {
        return make_float2(bf16_bits_to_float(this->w[i] & 0xffffu), __uint_as_float(this->w[i] & 0xffff0000u));
    }
    __device__ void put2(int i, float2 x) { this->w[i] = pack_bf16x2(x.x, x.y); }
};
template <int V>
struct alignas(2 * V) RopeVec<__half, V> : RopeVec16<__half, V> {
    __device__ float2 get2(int i) const { return __half22float2(*reinterpret_cast<const __half2 *>(&this->w[i])); }
    __device__ void put2(int i, float2 x) { this->w[i] = pack_f16x2(x.x, x.y); }
};
template <>
struct alignas(2) RopeVec<__nv_bfloat16, 1> {
    __nv_bfloat16 e;
    __device__ float get(int) const { return __bfloat162float(e); }
    __device__ void put(int, float x) { e = __float2bfloat16_rn(x); }
};
template <>
struct alignas(2) RopeVec<__half, 1> {
    __half e;
    __device__ float get(int) const { return __half2float(e); }
    __device__ void put(int, float x) { e = __float2half_rn(x); }
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
    else if (s > 64) turn = (hi >> (s - 64)) + ((hi >> (s - 65)) & 1);      // (rounded: the last bit shifted out)
    else if (s == 64) turn = hi + (lo >> 63);
    else if (s > 0) turn = ((hi << (64 - s)) | (lo >> s)) + ((lo >> (s - 1)) & 1);
    else if (s > -64) turn = lo << -s;
    uint64_t phase = turn * static_cast<uint64_t>(static_cast<int64_t>(position));
    if (bits >> 63) phase = 0 - phase;
    return __ll2float_rn(static_cast<int64_t>(phase)) * 0x1p-63f;
}

}  // namespace pa
