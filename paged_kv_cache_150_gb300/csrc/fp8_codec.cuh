// The 8-bit cache's number format: e4m3 codes with one power-of-two scale per
// (token, KV head) row, kept as a biased exponent byte.
//
// A row x of D values has the scale 2^e, e the smallest integer in
// [kScaleMin, kScaleMax] with |x_d| <= 448 * 2^e for its finite values (448 is
// the largest e4m3 value), and codes e4m3(x_d * 2^-e): a product by a power
// of two is exact, so a code is one rounding (nearest even) of the value and
// decoding in fp32 is exact.  e4m3 keeps its own exponent, so a finer scale
// than a power of two would gain at most one binade at the subnormal end; the
// byte costs 1 / D of the codes' traffic where an fp32 scale costs 4 / D.
// An infinity becomes +-448 * 2^e, a NaN stays one.
#pragma once

#include <cuda_fp8.h>

#include "pa_internal.h"

namespace pa {

constexpr int kScaleBias = 127, kScaleMin = -126, kScaleMax = 120;

// Scale exponent of a row whose largest finite |x| has the fp32 bits amax.
// amax = 1.f * 2^(E - 127) against 448 * 2^e = 1.75 * 2^(8 + e).
__device__ __forceinline__ int32_t row_exponent(uint32_t amax) {
    const int32_t E = (int32_t)(amax >> 23);
    const int32_t e = E - 135 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, kScaleMin);  // E <= 254: e <= 120
}
// |x| as fp32 bits, 0 for infinities and NaN (they set no scale).
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}
// 2^-e for e in [kScaleMin, kScaleMax] (a normal fp32 number).
__device__ __forceinline__ float inv_scale(int32_t e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// 2^(b - 127) of a scale byte b < 255; infinity for 255.
__device__ __forceinline__ float scale_bits(uint32_t b) { return __uint_as_float(max(b << 23, 0x00400000u)); }
// 2^(b - 127) of a scale byte b (255, which no write produces, is NaN).
__device__ __forceinline__ float scale_of(uint32_t b) { return b == 255 ? __uint_as_float(0x7fffffffu) : scale_bits(b); }

// Four e4m3 codes of a word, byte 0 first.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ float4 decode4(uint32_t w) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    return make_float4(a.x, a.y, b.x, b.y);
}

// The codes of a word's low and high half to fp16 (exact).
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// An 8-bit pool's descriptor: row layout, a scale per token or per block.
inline pa_status_t validate_fp8_desc(const pa_cache_desc_t *c) {
    if (!c) return PA_ERR_INVALID_ARG;
    if (c->num_blocks <= 0 || c->block_size <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0) return PA_ERR_INVALID_ARG;
    if (c->dtype != PA_FP8_E4M3 && c->dtype != PA_FP8_E4M3_BLOCK) return PA_ERR_INVALID_ARG;
    if (c->layout != PA_LAYOUT_ROW) return c->layout == PA_LAYOUT_SPLIT ? PA_ERR_UNSUPPORTED : PA_ERR_INVALID_ARG;
    if ((int64_t)c->num_blocks * c->block_size >= ((int64_t)1 << 31)) return PA_ERR_INVALID_ARG;
    if ((int64_t)c->num_kv_heads * c->head_dim >= ((int64_t)1 << 31)) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

}  // namespace pa
