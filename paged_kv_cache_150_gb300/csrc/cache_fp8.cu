// The 8-bit cache's write, read-back and block copy.
//
// Write: one pass over the new rows.  A row of D values (one token, one KV
// head) is held by a group of lanes, one 16-byte vector each where D allows;
// its largest |x| is a shuffle reduction within the group, then every lane
// encodes the values it still holds.  Read-back: one pass the other way.  Both
// are bound by HBM traffic (x once, codes and one scale byte once).
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
    // Largest finite |x| over the rows that L lanes hold of K and of V, as fp32 bits.
    template <int L>
    static __device__ __forceinline__ void row_max(const uint4 &k, const uint4 &v, uint32_t &ka, uint32_t &va) {
        auto lane_max = [](const uint4 &u) {
            return max(max(finite_bits(__uint_as_float(u.x)), finite_bits(__uint_as_float(u.y))),
                       max(finite_bits(__uint_as_float(u.z)), finite_bits(__uint_as_float(u.w))));
        };
        ka = lane_max(k), va = lane_max(v);
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
    // The same in 16-bit pairs: K's and V's maxima travel in one word.
    template <int L>
    static __device__ __forceinline__ void row_max(const uint4 &k, const uint4 &v, uint32_t &ka, uint32_t &va) {
        auto lane_max = [](const uint4 &u) {
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
        };
        uint32_t m = lane_max(k) << 16 | lane_max(v);
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

// Rows (write) and vectors (read) that a lane has in flight, of K and of V,
// and the CTAs of 256 threads resident per SM that its registers are held to.
constexpr int kWriteRows = 4, kWriteCtas = 4, kReadRows = 2, kReadCtas = 6;

// Write, fewer than 2^31 rows of at most 32 vectors.  Rows (t, h) are numbered
// t * Hk + h; L lanes (a power of two) hold a row, one vector each, a warp
// takes 32 / L rows at a time, kWriteRows passes at once, K and V together.
template <typename T, int L>
__global__ void __launch_bounds__(256, kWriteCtas) write_fp8_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                        const int32_t *__restrict__ slots, uint32_t rows, uint32_t Hk,
                                                        int32_t vecs, uint8_t *__restrict__ kc,
                                                        uint8_t *__restrict__ vc, uint8_t *__restrict__ ks,
                                                        uint8_t *__restrict__ vs, int64_t num_slots,
                                                        unsigned int *__restrict__ err) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int N = Vec16<T>::N, GW = 32 / L;
    const int lane = threadIdx.x & 31, li = lane % L;
    const uint32_t w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const uint32_t nw = (gridDim.x * blockDim.x) >> 5;
    const bool in_row = li < vecs;
    for (uint32_t r0 = w * (GW * kWriteRows); r0 < rows; r0 += nw * (GW * kWriteRows)) {
        uint4 ku[kWriteRows], vu[kWriteRows];
        int64_t dst[kWriteRows];  // row of the pool, -1: none
#pragma unroll
        for (int u = 0; u < kWriteRows; ++u) {
            const uint32_t r = r0 + u * GW + lane / L;
            dst[u] = -1;
            ku[u] = vu[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) {
                const uint32_t t = r / Hk;
                const int32_t s = __ldg(slots + t);
                if (s >= num_slots) {
                    if (li == 0) atomicOr(err, kErrBounds);
                } else if (s >= 0) {
                    dst[u] = (int64_t)s * Hk + (r - t * Hk);
                    if (in_row) {
                        ku[u] = __ldcs(reinterpret_cast<const uint4 *>(k) + (int64_t)r * vecs + li);
                        vu[u] = __ldcs(reinterpret_cast<const uint4 *>(v) + (int64_t)r * vecs + li);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kWriteRows; ++u) {
            uint32_t ka, va;
            Vec16<T>::template row_max<L>(ku[u], vu[u], ka, va);
            if (dst[u] >= 0) {
                float kx[N], vx[N];
                Vec16<T>::load(ku[u], kx);
                Vec16<T>::load(vu[u], vx);
                const int32_t ke = row_exponent(ka), ve = row_exponent(va);
                if (in_row) {
                    const int64_t at = (dst[u] * vecs + li) * N;
                    store_codes<N>(kc + at, kx, inv_scale(ke));
                    store_codes<N>(vc + at, vx, inv_scale(ve));
                }
                if (li == 0) {
                    ks[dst[u]] = (uint8_t)(ke + kScaleBias);
                    vs[dst[u]] = (uint8_t)(ve + kScaleBias);
                }
            }
        }
    }
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float *p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Write, any row length and alignment: one warp per row, two passes over it
// (the second finds it in L1 or L2), one element per lane at a time.
template <typename T>
__global__ void __launch_bounds__(256) write_fp8_any_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                            const int32_t *__restrict__ slots, int64_t rows,
                                                            int32_t Hk, int32_t D, uint8_t *__restrict__ kc,
                                                            uint8_t *__restrict__ vc, uint8_t *__restrict__ ks,
                                                            uint8_t *__restrict__ vs, int64_t num_slots,
                                                            unsigned int *__restrict__ err) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t nw = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; r < rows; r += nw) {
        const int64_t t = r / Hk;
        const int32_t s = __ldg(slots + t);
        if (s < 0) continue;
        if (s >= num_slots) {
            if (lane == 0) atomicOr(err, kErrBounds);
            continue;
        }
        const int64_t dst = (int64_t)s * Hk + (r - t * Hk);
        uint32_t ka = 0, va = 0;
        for (int32_t d = lane; d < D; d += 32) {
            ka = max(ka, finite_bits(to_f32(k[r * D + d])));
            va = max(va, finite_bits(to_f32(v[r * D + d])));
        }
        ka = __reduce_max_sync(0xffffffffu, ka);
        va = __reduce_max_sync(0xffffffffu, va);
        const int32_t ke = row_exponent(ka), ve = row_exponent(va);
        const float ki = inv_scale(ke), vi = inv_scale(ve);
        for (int32_t d = lane; d < D; d += 32) {
            kc[dst * D + d] = (uint8_t)__nv_cvt_float_to_fp8(to_f32(k[r * D + d]) * ki, __NV_SATFINITE, __NV_E4M3);
            vc[dst * D + d] = (uint8_t)__nv_cvt_float_to_fp8(to_f32(v[r * D + d]) * vi, __NV_SATFINITE, __NV_E4M3);
        }
        if (lane == 0) {
            ks[dst] = (uint8_t)(ke + kScaleBias);
            vs[dst] = (uint8_t)(ve + kScaleBias);
        }
    }
}

// Read-back, D a multiple of the 16-byte output vector's elements and fewer
// than 2^31 vectors: one output vector per thread and pass, kReadRows passes of
// K and V in flight.
template <typename T>
__global__ void __launch_bounds__(256, kReadCtas) read_fp8_kernel(T *__restrict__ k, T *__restrict__ v,
                                                       const int32_t *__restrict__ slots, uint32_t total, uint32_t Hk,
                                                       uint32_t vecs, const uint8_t *__restrict__ kc,
                                                       const uint8_t *__restrict__ vc, const uint8_t *__restrict__ ks,
                                                       const uint8_t *__restrict__ vs, int64_t num_slots,
                                                       unsigned int *__restrict__ err) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int N = Vec16<T>::N;
    using Code = typename std::conditional<N == 8, uint2, uint32_t>::type;
    const uint32_t stride = gridDim.x * blockDim.x;
    for (uint32_t i0 = blockIdx.x * blockDim.x + threadIdx.x; i0 < total; i0 += stride * kReadRows) {
        Code kq[kReadRows], vq[kReadRows];
        uint32_t kb[kReadRows], vb[kReadRows];
#pragma unroll
        for (int u = 0; u < kReadRows; ++u) {
            const uint32_t i = i0 + u * stride;
            kq[u] = Code{}, vq[u] = Code{};  // padding and bad slots decode to zeros
            kb[u] = vb[u] = kScaleBias;
            if (i < total) {
                const uint32_t r = i / vecs, t = r / Hk, c = i - r * vecs;
                const int32_t s = __ldg(slots + t);
                if (s >= num_slots) {
                    if (c == 0) atomicOr(err, kErrBounds);
                } else if (s >= 0) {
                    const int64_t src = (int64_t)s * Hk + (r - t * Hk);
                    kq[u] = __ldcs(reinterpret_cast<const Code *>(kc) + src * vecs + c);
                    vq[u] = __ldcs(reinterpret_cast<const Code *>(vc) + src * vecs + c);
                    kb[u] = __ldg(ks + src);
                    vb[u] = __ldg(vs + src);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kReadRows; ++u) {
            const uint32_t i = i0 + u * stride;
            if (i >= total) break;
            auto emit = [&](const Code &q, uint32_t b, T *out) {
                const float s = scale_of(b);
                float x[N];
                if constexpr (N == 8) {
                    const float4 lo = decode4(q.x), hi = decode4(q.y);
                    x[0] = lo.x * s, x[1] = lo.y * s, x[2] = lo.z * s, x[3] = lo.w * s;
                    x[4] = hi.x * s, x[5] = hi.y * s, x[6] = hi.z * s, x[7] = hi.w * s;
                } else {
                    const float4 lo = decode4(q);
                    x[0] = lo.x * s, x[1] = lo.y * s, x[2] = lo.z * s, x[3] = lo.w * s;
                }
                __stcs(reinterpret_cast<uint4 *>(out) + i, Vec16<T>::pack(x));
            };
            emit(kq[u], kb[u], k);
            emit(vq[u], vb[u], v);
        }
    }
}

// Read-back, any row length and alignment: one element per thread.
template <typename T>
__global__ void __launch_bounds__(256) read_fp8_any_kernel(T *__restrict__ k, T *__restrict__ v,
                                                           const int32_t *__restrict__ slots, int64_t total,
                                                           int32_t Hk, int32_t D, const uint8_t *__restrict__ kc,
                                                           const uint8_t *__restrict__ vc,
                                                           const uint8_t *__restrict__ ks,
                                                           const uint8_t *__restrict__ vs, int64_t num_slots,
                                                           unsigned int *__restrict__ err) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
        const int64_t r = i / D, t = r / Hk;
        const int32_t d = (int32_t)(i - r * D);
        const int32_t s = __ldg(slots + t);
        float kx = 0.f, vx = 0.f;
        if (s >= num_slots) {
            if (d == 0) atomicOr(err, kErrBounds);
        } else if (s >= 0) {
            const int64_t src = (int64_t)s * Hk + (r - t * Hk);
            kx = decode4(kc[src * D + d]).x * scale_of(ks[src]);
            vx = decode4(vc[src * D + d]).x * scale_of(vs[src]);
        }
        from_f32(k + i, kx);
        from_f32(v + i, vx);
    }
}

namespace {

// Work's CTAs, at most per_sm per SM (one wave).
int grid_for(int64_t ctas, int per_sm) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)std::max(num_sms(), 1) * per_sm));
}
// The vector kernels count in 32 bits, with room for one grid stride past the end.
constexpr int64_t kIndexMax = (int64_t)1 << 31;

template <typename T>
bool aligned_rows(int32_t D, const void *x, const void *y, const void *a, const void *b) {
    constexpr int N = Vec16<T>::N;
    return D % N == 0 && (((uintptr_t)x | (uintptr_t)y) & 15) == 0 && (((uintptr_t)a | (uintptr_t)b) & (N - 1)) == 0;
}

template <typename T>
cudaError_t launch_write(const T *k, const T *v, const int32_t *slots, int32_t T_, uint8_t *kc, uint8_t *vc, uint8_t *ks,
                         uint8_t *vs, const pa_cache_desc_t *c, unsigned int *err, cudaStream_t s) {
    int64_t rows = (int64_t)T_ * c->num_kv_heads, ns = (int64_t)c->num_blocks * c->block_size;
    int32_t Hk = c->num_kv_heads, D = c->head_dim, vecs = D / Vec16<T>::N;
    if (!aligned_rows<T>(D, k, v, kc, vc) || vecs > 32 || rows >= kIndexMax) {
        void *args[] = {&k, &v, &slots, &rows, &Hk, &D, &kc, &vc, &ks, &vs, &ns, &err};
        return launch_pdl((const void *)write_fp8_any_kernel<T>, dim3(grid_for((rows + 7) / 8, 8)), dim3(256), args, 0, s);
    }
    int L = 1;
    while (L < vecs) L *= 2;
    const void *fn = L == 32  ? (const void *)write_fp8_kernel<T, 32>
                     : L == 16 ? (const void *)write_fp8_kernel<T, 16>
                     : L == 8  ? (const void *)write_fp8_kernel<T, 8>
                     : L == 4  ? (const void *)write_fp8_kernel<T, 4>
                     : L == 2  ? (const void *)write_fp8_kernel<T, 2>
                               : (const void *)write_fp8_kernel<T, 1>;
    const int64_t per_cta = 8 * (32 / L) * kWriteRows;
    uint32_t rows32 = (uint32_t)rows;
    void *args[] = {&k, &v, &slots, &rows32, &Hk, &vecs, &kc, &vc, &ks, &vs, &ns, &err};
    return launch_pdl(fn, dim3(grid_for((rows + per_cta - 1) / per_cta, kWriteCtas)), dim3(256), args, 0, s);
}

template <typename T>
cudaError_t launch_read(T *k, T *v, const int32_t *slots, int32_t T_, const uint8_t *kc, const uint8_t *vc,
                        const uint8_t *ks, const uint8_t *vs, const pa_cache_desc_t *c, unsigned int *err,
                        cudaStream_t s) {
    int64_t ns = (int64_t)c->num_blocks * c->block_size;
    int32_t Hk = c->num_kv_heads, D = c->head_dim, vecs = D / Vec16<T>::N;
    if (!aligned_rows<T>(D, k, v, kc, vc) || (int64_t)T_ * Hk * vecs >= kIndexMax) {
        int64_t total = (int64_t)T_ * Hk * D;
        void *args[] = {&k, &v, &slots, &total, &Hk, &D, &kc, &vc, &ks, &vs, &ns, &err};
        return launch_pdl((const void *)read_fp8_any_kernel<T>, dim3(grid_for((total + 255) / 256, 8)), dim3(256), args, 0, s);
    }
    uint32_t total = (uint32_t)((int64_t)T_ * Hk * vecs);
    void *args[] = {&k, &v, &slots, &total, &Hk, &vecs, &kc, &vc, &ks, &vs, &ns, &err};
    // fp32 rows, four bytes out for one in, run faster one pass per thread, bf16
    // rows on one wave, at every size measured (us; one pass, one wave):
    //   tokens x heads x D    fp32           bf16
    //     5000 x 8 x 128       10.9   11.8     8.6    8.8
    //    20000 x 8 x 128       33.7   36.6    22.5   21.7
    //   131072 x 8 x 128      213.1  221.4   135.7  125.0
    //   131072 x 8 x 64       106.1  111.0    69.7   63.3
    //   131072 x 1 x 128       29.3   31.2    20.8   18.7
    //    60000 x 8 x 256      191.7  205.1   122.4  118.5
    const int64_t ctas = ((int64_t)total + 256 * kReadRows - 1) / (256 * kReadRows);
    const int grid = sizeof(T) == 4 ? (int)ctas : grid_for(ctas, kReadCtas);
    return launch_pdl((const void *)read_fp8_kernel<T>, dim3(grid), dim3(256), args, 0, s);
}

pa_status_t check_rows_call(const pa_cache_desc_t *cache, int32_t num_tokens, int32_t dtype) {
    const pa_status_t st = validate_fp8_desc(cache);
    if (st != PA_OK) return st;
    if (num_tokens < 0 || (dtype != PA_F32 && dtype != PA_BF16)) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status_t pa_reshape_and_cache_fp8(const void *k, const void *v, int32_t dtype, const int32_t *slot_mapping,
                                                int32_t num_tokens, void *k_cache, void *v_cache, uint8_t *k_scale,
                                                uint8_t *v_scale, const pa_cache_desc_t *cache, pa_stream_t stream) try {
    const pa_status_t st = check_rows_call(cache, num_tokens, dtype);
    if (st != PA_OK) return st;
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache || !k_scale || !v_scale) return PA_ERR_INVALID_ARG;
    if (((uintptr_t)k | (uintptr_t)v) % (size_t)dtype_bytes(dtype) != 0) return PA_ERR_INVALID_ARG;
    unsigned int *err = device_error_word();
    if (!err) return PA_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    cudaGetLastError();
    const cudaError_t e =
        dtype == PA_BF16
            ? launch_write((const __nv_bfloat16 *)k, (const __nv_bfloat16 *)v, slot_mapping, num_tokens,
                           (uint8_t *)k_cache, (uint8_t *)v_cache, k_scale, v_scale, cache, err, s)
            : launch_write((const float *)k, (const float *)v, slot_mapping, num_tokens, (uint8_t *)k_cache,
                           (uint8_t *)v_cache, k_scale, v_scale, cache, err, s);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
} catch (...) {
    return host_failure();
}

extern "C" pa_status_t pa_gather_cache_fp8(void *k, void *v, int32_t dtype, const int32_t *slot_mapping,
                                           int32_t num_tokens, const void *k_cache, const void *v_cache,
                                           const uint8_t *k_scale, const uint8_t *v_scale,
                                           const pa_cache_desc_t *cache, pa_stream_t stream) try {
    const pa_status_t st = check_rows_call(cache, num_tokens, dtype);
    if (st != PA_OK) return st;
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache || !k_scale || !v_scale) return PA_ERR_INVALID_ARG;
    if (((uintptr_t)k | (uintptr_t)v) % (size_t)dtype_bytes(dtype) != 0) return PA_ERR_INVALID_ARG;
    unsigned int *err = device_error_word();
    if (!err) return PA_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    cudaGetLastError();
    const cudaError_t e =
        dtype == PA_BF16 ? launch_read((__nv_bfloat16 *)k, (__nv_bfloat16 *)v, slot_mapping, num_tokens,
                                       (const uint8_t *)k_cache, (const uint8_t *)v_cache, k_scale, v_scale, cache, err, s)
                         : launch_read((float *)k, (float *)v, slot_mapping, num_tokens, (const uint8_t *)k_cache,
                                       (const uint8_t *)v_cache, k_scale, v_scale, cache, err, s);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
} catch (...) {
    return host_failure();
}

extern "C" pa_status_t pa_copy_blocks_fp8(void *k_cache, void *v_cache, uint8_t *k_scale, uint8_t *v_scale,
                                          const pa_cache_desc_t *cache, const int32_t *src_dst_pairs,
                                          int32_t num_pairs, pa_stream_t stream) try {
    const pa_status_t st = validate_fp8_desc(cache);
    if (st != PA_OK) return st;
    if (num_pairs < 0) return PA_ERR_INVALID_ARG;
    if (num_pairs == 0) return PA_OK;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !src_dst_pairs) return PA_ERR_INVALID_ARG;
    unsigned int *err = device_error_word();
    if (!err) return PA_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    cudaGetLastError();
    const int64_t rows = (int64_t)cache->block_size * cache->num_kv_heads;
    launch_copy_blocks(k_cache, v_cache, rows * cache->head_dim, cache->num_blocks, src_dst_pairs, num_pairs, err, s);
    launch_copy_blocks(k_scale, v_scale, rows, cache->num_blocks, src_dst_pairs, num_pairs, err, s);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
} catch (...) {
    return host_failure();
}
