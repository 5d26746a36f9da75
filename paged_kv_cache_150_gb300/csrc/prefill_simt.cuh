// Chunk attention on the CUDA cores (pa_prefill for fp32, head_dim 256, the
// split layout and block sizes the tensor-core kernel does not take; and the
// single queries of pa_decode_fp8 in the same cases).
//
// One CTA of 256 threads holds a tile of 64 query rows (64 / G tokens x the G
// heads of one KV head) and walks its units of 64 keys: S = Q K^T with 4 x 4
// scores per thread, the online softmax of each row in the 16 threads that
// share it, O += P V with 4 x (D / 16) accumulators per thread.  All
// arithmetic is fp32 (8-bit codes are decoded, bf16 widened, as a tile is
// staged).  Per four steps of the head dimension a thread makes 64 FMAs from
// 8 16-byte shared loads (4 of them broadcasts); the shared-memory wavefronts bound
// it (73% of their peak, FMA pipes 51%: six fp32 chunks of 61 to 331 tokens over
// contexts of up to 1500, 32 heads, head_dim 64, 238 us).
// fp32 rows of head_dim 64 and 128 are staged by cp.async a unit ahead, into
// the second of two buffers, with the block-table entries read two units
// ahead; the other kinds are staged in place.
#pragma once

#include <type_traits>

#include "fp8_codec.cuh"
#include "prefill_plan.cuh"

namespace pa {

// Element kinds of a cache, as the kernels read them.
struct CacheE4m3 {};

constexpr int kSimtRows = 64, kSimtKeys = 64, kSimtThreads = 256, kSimtExtra = 1;

// Shared memory: Q and K tiles with rows of D + 4 floats (rows of a 16-byte
// column fall in distinct banks), V rows of D, P rows of 64 + 4, and the
// element offset of each key's row.
template <int D, bool kPipe>
struct SimtSmem {
    static constexpr int kBufs = kPipe ? 2 : 1;
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kSimtRows * (D + 4);
    static constexpr int kV = kK + kBufs * kSimtKeys * (D + 4);
    static constexpr int kP = kV + kBufs * kSimtKeys * D;
    static constexpr int kSlots = kP + kSimtRows * (kSimtKeys + 4);
    static constexpr size_t kBytes = (size_t)kSlots * 4 + kBufs * kSimtKeys * 8;
};
// Whether a kind of cache is staged ahead.
template <typename CT, int D, int LAYOUT>
constexpr bool simt_pipe() {
    return std::is_same<CT, float>::value && LAYOUT == PA_LAYOUT_ROW && D <= 128;
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

// Four elements at d (a multiple of 4) of the K or V row of slot `slot`, KV
// head kvh.  CT: float, __nv_bfloat16 or CacheE4m3 (row layout only).
template <typename CT, int D, int LAYOUT, bool IS_V>
__device__ __forceinline__ float4 cache4(const PrefillArgs &a, int64_t slot, int32_t kvh, int d) {
    const void *base = IS_V ? a.v_cache : a.k_cache;
    if constexpr (std::is_same<CT, CacheE4m3>::value) {
        const int64_t row = slot * a.Hk + kvh;
        const float s = scale_of(__ldg((IS_V ? a.v_scale : a.k_scale) + row));
        const float4 x = decode4(__ldg(reinterpret_cast<const uint32_t *>((const uint8_t *)base + row * D + d)));
        return make_float4(x.x * s, x.y * s, x.z * s, x.w * s);
    } else if constexpr (LAYOUT == PA_LAYOUT_ROW) {
        return load4((const CT *)base + (slot * a.Hk + kvh) * D + d);
    } else {
        const int64_t blk = slot / a.B, off = slot - blk * a.B, head = blk * a.Hk + kvh;
        constexpr int X = 16 / (int)sizeof(CT);
        if constexpr (!IS_V) return load4((const CT *)base + ((head * (D / X) + d / X) * a.B + off) * X + d % X);
        const CT *p = (const CT *)base + (head * D + d) * a.B + off;
        return make_float4((float)p[0], (float)p[a.B], (float)p[2 * (int64_t)a.B], (float)p[3 * (int64_t)a.B]);
    }
}

// Whether 4-element accesses to q are aligned; without it the rows are read
// element by element (q and out are only 2-element aligned by contract).
template <typename T>
__device__ __forceinline__ float4 load4_any(const T *p) {
    if (((uintptr_t)p & (4 * sizeof(T) - 1)) == 0) return load4(p);
    return make_float4((float)p[0], (float)p[1], (float)p[2], (float)p[3]);
}

// O += P V over the staged unit for this thread's 4 rows and D / 16 columns
// (tx * 4 + 64 w); kSeen: each row adds the keys it sees only.
template <bool kSeen, int EV>
__device__ __forceinline__ void add_pv(const float *Ps, const float *Vs, float (&o)[4][EV * 4], int ty, int tx,
                                       int32_t key0, const int32_t (&last)[4]) {
    constexpr int D = EV * 64, PS = kSimtKeys + 4;
#pragma unroll 2
    for (int k4 = 0; k4 < kSimtKeys; k4 += 4) {
        float4 px[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) px[i] = *reinterpret_cast<const float4 *>(Ps + (ty * 4 + i) * PS + k4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
            for (int w = 0; w < EV; ++w) {
                const float4 vx = *reinterpret_cast<const float4 *>(Vs + (k4 + kk) * D + 64 * w + tx * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (kSeen && key0 + k4 + kk > last[i]) continue;
                    const float p = kk == 0 ? px[i].x : kk == 1 ? px[i].y : kk == 2 ? px[i].z : px[i].w;
                    o[i][4 * w] = fmaf(p, vx.x, o[i][4 * w]);
                    o[i][4 * w + 1] = fmaf(p, vx.y, o[i][4 * w + 1]);
                    o[i][4 * w + 2] = fmaf(p, vx.z, o[i][4 * w + 2]);
                    o[i][4 * w + 3] = fmaf(p, vx.w, o[i][4 * w + 3]);
                }
            }
        }
    }
}

template <typename T, typename CT, int D, int LAYOUT>
__global__ void __launch_bounds__(kSimtThreads, D == 256 ? 1 : 2)
    prefill_simt_kernel(const __grid_constant__ PrefillArgs a) {
    constexpr bool kPipe = simt_pipe<CT, D, LAYOUT>();
    using L = SimtSmem<D, kPipe>;
    extern __shared__ __align__(16) float sm[];
    float *Qs = sm + L::kQ, *Ps = sm + L::kP;
    int64_t *slots = reinterpret_cast<int64_t *>(sm + L::kSlots);
    constexpr int QS = D + 4, PS = kSimtKeys + 4, EV = D / 64;  // row strides, float4 columns per thread
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t c = blockIdx.x;
    PrefillCursor cur;
    const bool work = cur.init(a, c);
    if (tid == 0) note_cut(a, c, work, cur);
    if (!work) return;
    do {
        const PrefillTile t = cur.t;
        const int32_t nrow = t.ntok * a.G;  // rows of this tile (<= 64)
        const int32_t keys = t.p0 + t.ntok, j0 = cur.j0, j1 = cur.j1;
        const int32_t *row = a.tables + (int64_t)t.seq * a.max_blocks;
        // Thread i < 64: the table entry of key i of unit j (0 without that
        // key), and the slot it makes (-1: no key, or a bad entry: zeros).
        auto entry = [&](int32_t j) -> int32_t {
            const int64_t pos = (int64_t)j * kSimtKeys + tid;
            return tid < kSimtKeys && j < j1 && pos < keys ? row[pos / a.B] : 0;
        };
        auto put_slot = [&](int32_t j, int32_t phys) {
            if (tid >= kSimtKeys || j >= j1) return;
            const int64_t pos = (int64_t)j * kSimtKeys + tid;
            int64_t slot = -1;
            if (pos < keys) {
                if (phys < 0 || phys >= a.NB)
                    atomicOr(a.err, kErrBounds);
                else
                    slot = (int64_t)phys * a.B + pos % a.B;
            }
            slots[(kPipe ? (j & 1) * kSimtKeys : 0) + tid] = slot;
        };
        auto k_buf = [&](int32_t j) { return sm + L::kK + (kPipe ? (j & 1) * kSimtKeys * QS : 0); };
        auto v_buf = [&](int32_t j) { return sm + L::kV + (kPipe ? (j & 1) * kSimtKeys * D : 0); };
        // K and V rows of unit j into its buffers (kPipe: asynchronously).
        auto stage = [&](int32_t j) {
            const int64_t *sl = slots + (kPipe ? (j & 1) * kSimtKeys : 0);
            float *Ks = k_buf(j), *Vs = v_buf(j);
            for (int e = tid; e < kSimtKeys * (D / 4); e += kSimtThreads) {
                const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
                const int64_t slot = sl[r];
                if (kPipe && slot >= 0) {
                    const int64_t at = (slot * a.Hk + cur.kvh) * D + d;
                    cp_async16(Ks + r * QS + d, (const float *)a.k_cache + at);
                    cp_async16(Vs + r * D + d, (const float *)a.v_cache + at);
                } else {
                    float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
                    if (slot >= 0) {
                        kx = cache4<CT, D, LAYOUT, false>(a, slot, cur.kvh, d);
                        vx = cache4<CT, D, LAYOUT, true>(a, slot, cur.kvh, d);
                    }
                    *reinterpret_cast<float4 *>(Ks + r * QS + d) = kx;
                    *reinterpret_cast<float4 *>(Vs + r * D + d) = vx;
                }
            }
            if (kPipe) cp_async_commit();
        };
        int32_t phys = entry(j0), phys_next = kPipe ? entry(j0 + 1) : 0;
        __syncthreads();  // the previous segment's reads of shared memory
        for (int e = tid; e < kSimtRows * (D / 4); e += kSimtThreads) {
            const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < nrow) {
                const int tok = r / a.G, g = r - tok * a.G;
                x = load4_any((const T *)a.q + ((int64_t)(t.row0 + tok) * a.H + (int64_t)cur.kvh * a.G + g) * D + d);
            }
            *reinterpret_cast<float4 *>(Qs + r * QS + d) = x;
        }
        if (kPipe) {
            put_slot(j0, phys);
            put_slot(j0 + 1, phys_next);
            __syncthreads();
            stage(j0);
        }
        float o[4][EV * 4], m[4], l[4];
        int32_t last[4];  // this thread's rows: last key position each sees
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            last[i] = r < nrow ? t.p0 + r / a.G : -1;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < EV * 4; ++e) o[i][e] = 0.f;
        }
        for (int32_t j = j0; j < j1; ++j) {
            const int32_t key0 = j * kSimtKeys;
            if (kPipe) {
                if (j > j0) __syncthreads();  // the last unit's reads of the other buffers are done, slots of j + 1 written
                if (j + 1 < j1) stage(j + 1);
                phys = entry(j + 2);
                if (j + 1 < j1)
                    cp_async_wait<1>();
                else
                    cp_async_wait<0>();
            } else {
                if (j > j0) __syncthreads();
                put_slot(j, phys);
                if (j + 1 < j1) phys = entry(j + 1);
                __syncthreads();
                stage(j);
            }
            const float *Ks = k_buf(j), *Vs = v_buf(j);
            __syncthreads();  // unit j staged
            // Keys that only some rows see: does V hold a value that is not finite?
            bool bad = false;
            if (t.p0 + 1 - key0 < kSimtKeys) {  // (key0 + kSimtKeys may pass 2^31)
                bool odd = false;
                for (int e = tid; e < kSimtKeys * (D / 4); e += kSimtThreads) {
                    const float4 vx = *reinterpret_cast<const float4 *>(Vs + e * 4);
                    // a product with 0 is NaN exactly where an element is not finite
                    odd = odd || vx.x * 0.f + vx.y * 0.f + (vx.z * 0.f + vx.w * 0.f) != 0.f;
                }
                bad = __syncthreads_or(odd) != 0;
            }
            // S: rows ty * 4 + i, keys tx + 16 * n
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < 4; ++n) s[i][n] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 qx[4], kx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) qx[i] = *reinterpret_cast<const float4 *>(Qs + (ty * 4 + i) * QS + d);
#pragma unroll
                for (int n = 0; n < 4; ++n) kx[n] = *reinterpret_cast<const float4 *>(Ks + (tx + 16 * n) * QS + d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        s[i][n] = fmaf(qx[i].x, kx[n].x, s[i][n]);
                        s[i][n] = fmaf(qx[i].y, kx[n].y, s[i][n]);
                        s[i][n] = fmaf(qx[i].z, kx[n].z, s[i][n]);
                        s[i][n] = fmaf(qx[i].w, kx[n].w, s[i][n]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    s[i][n] = key0 + tx + 16 * n <= last[i] ? s[i][n] * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[i][n]);
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                const float mn = fmaxf(m[i], mx), mref = mn == -INFINITY ? 0.f : mn;  // no key yet: zeros
                const float al = ex2_approx(m[i] - mref);
                m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float p = ex2_approx(s[i][n] - mref);
                    sum += p;
                    Ps[(ty * 4 + i) * PS + tx + 16 * n] = p;
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                l[i] = l[i] * al + sum;
#pragma unroll
                for (int e = 0; e < EV * 4; ++e) o[i][e] *= al;
            }
            __syncwarp();  // a row's scores stay within its warp (2 values of ty)
            // Keys that a row does not see carry p = 0 exactly, but 0 x V is
            // not 0 where V is not finite (a later token of the chunk): a
            // unit with such a value takes the sums over seen keys only.
            if (!bad)
                add_pv<false, EV>(Ps, Vs, o, ty, tx, key0, last);
            else
                add_pv<true, EV>(Ps, Vs, o, ty, tx, key0, last);
            if (kPipe) put_slot(j + 2, phys);  // its buffer's slots were read when unit j was staged
        }
        const bool whole = cur.whole();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= nrow) continue;
            if (whole) {
                const int tok = r / a.G, g = r - tok * a.G;
                const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
                T *op = (T *)a.out + ((int64_t)(t.row0 + tok) * a.H + (int64_t)cur.kvh * a.G + g) * D + tx * 4;
#pragma unroll
                for (int w = 0; w < EV; ++w)
#pragma unroll
                    for (int e = 0; e < 4; ++e) store_out(op + 64 * w + e, o[i][4 * w + e] * inv);
            } else {
                const int64_t row_p = cur.slot(c) * kSimtRows + r;
                float *ap = a.acc + row_p * D + tx * 4;
#pragma unroll
                for (int w = 0; w < EV; ++w)
                    *reinterpret_cast<float4 *>(ap + 64 * w) =
                        make_float4(o[i][4 * w], o[i][4 * w + 1], o[i][4 * w + 2], o[i][4 * w + 3]);
                if (tx == 0) a.ml[row_p] = make_float2(m[i], l[i]);
            }
        }
    } while (cur.next(a));
}

}  // namespace pa
