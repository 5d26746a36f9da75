// Rows of new K and V on their way into an 8-bit cache and back: 16-byte
// vectors, their largest values, their codes.
#pragma once

#include "fp8_codec.cuh"

namespace pa {

// A group's 16 bytes of a row in fp32.
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z),
        x[3] = __uint_as_float(u.w);
    }
    // Largest finite |x| of a vector, in a form that compares by size; its fp32 bits.
    static __device__ __forceinline__ uint32_t largest(const uint4 &u) {
        return max(max(finite_bits(__uint_as_float(u.x)), finite_bits(__uint_as_float(u.y))),
                   max(finite_bits(__uint_as_float(u.z)), finite_bits(__uint_as_float(u.w))));
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
    // Largest finite |x| over the rows that L lanes hold of K and of V, as fp32 bits.
    template <int L>
    static __device__ __forceinline__ void row_max(const uint4 &k, const uint4 &v, uint32_t &ka, uint32_t &va) {
        ka = largest(k), va = largest(v);
        if constexpr (L == 32) {
            ka = __reduce_max_sync(0xffffffffu, ka);
            va = __reduce_max_sync(0xffffffffu, va);
        } else {
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                ka = max(ka, __shfl_xor_sync(0xffffffffu, ka, o));
                va = max(va, __shfl_xor_sync(0xffffffffu, va, o));
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // Largest finite |x| of a vector as bf16 bits; its fp32 bits.
    static __device__ __forceinline__ uint32_t largest(const uint4 &u) {
        const uint32_t w[4] = {u.x & 0x7fff7fffu, u.y & 0x7fff7fffu, u.z & 0x7fff7fffu, u.w & 0x7fff7fffu};
        uint32_t m = 0, odd = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = __vmaxu2(m, w[i]);
            odd |= (w[i] + 0x00800080u) & 0x80008000u;  // an exponent of all ones
        }
        if (odd) {
            m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & ~__vcmpgeu2(w[i], 0x7f807f80u));
        }
        return max(m >> 16, m & 0xffffu);
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m << 16; }
    // The same in 16-bit pairs: K's and V's maxima travel in one word.
    template <int L>
    static __device__ __forceinline__ void row_max(const uint4 &k, const uint4 &v, uint32_t &ka, uint32_t &va) {
        uint32_t m = largest(k) << 16 | largest(v);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        ka = m & 0xffff0000u, va = m << 16;
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};

// N codes (one vector's) to and from memory.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&x)[N], float inv) {
    if constexpr (N == 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(encode4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                                                   encode4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
    } else {
        *reinterpret_cast<uint32_t *>(p) = encode4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    }
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float *p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Work's CTAs, at most per_sm per SM (one wave).
inline int grid_for(int64_t ctas, int per_sm) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)std::max(num_sms(), 1) * per_sm));
}
template <typename T>
bool aligned_rows(int32_t D, const void *x, const void *y, const void *a, const void *b) {
    constexpr int N = Vec16<T>::N;
    return D % N == 0 && (((uintptr_t)x | (uintptr_t)y) & 15) == 0 && (((uintptr_t)a | (uintptr_t)b) & (N - 1)) == 0;
}

}  // namespace pa
