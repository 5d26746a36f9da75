// Tensor-core decode over the 8-bit cache (pa_decode_fp8 for head_dim 64 and
// 128, block sizes that are multiples of 8).
//
// What is computed: pa_decode's attention over K = 2^ek k8, V = 2^ev v8 with
// one exponent per token and KV head.  The codes are multiplied as fp16, which
// holds every e4m3 value exactly, on mma.sync (single queries: 8 heads or less
// per KV head, a contraction too thin for tcgen05's 128 rows):
//   S^T (16 tokens x 8 heads) = k8 Q^T, Q in fp16 scaled per row by a power of
//     two so that its largest element lies in [2^14, 2^15): exact for every
//     element within 2^28 of it;
//   x = S 2^ek 2^eq scale log2(e);
//   p = 2^(x - m), l += p,  O^T += v8^T P^T with P = p 2^(ev + m - m') in fp16.
// V's exponent goes into P, whose reference m' lies kTopBits below the running
// maximum of x + ev (m is that of x), so P's largest value stays within [2^7, 2^15]
// whatever the rows' sizes, near the top of fp16's range; at the end O is scaled
// by 2^(m' - m).  P is rounded to fp16 because the product takes it so: a relative
// 2^-11, or, of a P below 2^-14 (2^-21 of the largest), an absolute 2^-25 (2^-32
// of the largest; below that it counts as 0).  Over L keys the second kind adds
// up to at most L 2^-32 of the largest p |v|; with the reference at the maximum
// itself it was L 2^-25, more than the output's own rounding from 2^16 keys on.
// It is the only rounding beside fp32's and the output's.
//
// Bound by the K and V bytes: 16 sequences of 32768 tokens (64 / 8 heads, head_dim
// 128) take 169 to 174 us (6.2 to 6.4 TB/s) with the work list and the merge. The
// same bytes with 4 / 2 / 1 KV heads 174 / 181 / 221 us; head_dim 64 reaches 4.2 to
// 4.7 TB/s with 8 KV heads and 2.7 with one.  A CTA is 8 consumer warps and a TMA producer,
// two CTAs per SM; a stage is 8 slices of 16 tokens of one KV head (K and V,
// 32 KiB at head_dim 128): NH heads (the largest of 8, 4, 2, 1 that divides Hk)
// x 128 / NH tokens, so that a stage is one contiguous piece of every block it
// touches.  Warp w takes head w % NH, tokens 16 (w / NH) ...; with NH < 8 the
// warps of a head join their parts in shared memory at a segment's end.
// A fragment's order along a contraction is free: an ldmatrix of 16-bit units
// hands a thread 4 consecutive codes of a K row (Q is loaded in the same
// order), or of V (transposed) two tokens' codes of a pair of columns.
#pragma once

#include <cuda.h>  // CUtensorMap
#include <cuda_fp16.h>

#include "decode_merge.cuh"
#include "fp8_codec.cuh"
#include "prefill_plan.cuh"

namespace pa {

constexpr int kF8Warps = 8, kF8Threads = 32 * (kF8Warps + 1);
constexpr int kF8SlotRows = 64;  // query rows of a piece: NH * G <= 64
constexpr float kTopP = 256.f;   // 2^kLazyMaxSlack
constexpr float kTopBits = 7.f;  // P's reference below the running maximum: P <= 2^(7 + kLazyMaxSlack) < 65504
constexpr float kTopScale = 1.f / 128.f;  // 2^-kTopBits
constexpr float kMaxFactor = 3.4e38f;  // of p: just under fp32's end
constexpr int kF8Extra = 2;      // weight of a sequence beside its units (prefill_plan.cuh)

// The parts of a call beyond PrefillArgs (there G is NH * G and Hk the number
// of head groups).
struct F8Args {
    int32_t Hk, G, NH, T;   // KV heads, query heads per KV head, KV heads and tokens of a stage
    int32_t gran;           // tokens of a box: gcd(block size, T)
    int32_t stages;
    uint32_t scale_bytes;   // of K (or V) per stage: T * Hk
};

template <int D>
struct F8Smem {
    static constexpr uint32_t kTile = kF8Warps * 16 * D;  // K or V of a stage
    static constexpr uint32_t kJoinCols = 64;             // columns joined at a time
    // [stages][K tile, V tile] [stages][K scales, V scales] [barriers] [join]
    static __host__ __device__ uint32_t scales(int stages) { return (uint32_t)stages * 2 * kTile; }
    static __host__ __device__ uint32_t bars(int stages, uint32_t scale_bytes) {
        return (scales(stages) + (uint32_t)stages * 2 * scale_bytes + 15u) & ~15u;
    }
    static __host__ __device__ uint32_t join(int stages, uint32_t scale_bytes) {
        return (bars(stages, scale_bytes) + (uint32_t)stages * 16 + 15u) & ~15u;
    }
    // [kF8Warps - NH][G][kJoinCols] accumulators and [..][G] (m, l)
    static __host__ __device__ size_t bytes(int stages, uint32_t scale_bytes, int NH, int G) {
        return join(stages, scale_bytes) + (size_t)(kF8Warps - NH) * G * (kJoinCols * 4 + 8) + 1024;
    }
};

__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const void *tmap, uint32_t bar, int32_t c0, int32_t c1,
                                                 int32_t c2, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(tmap), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}
// bytes and both addresses are multiples of 16
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// The codes of a word's low and high half to fp16 (exact).
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Units of T tokens that the current segment takes: [j0, j1), none without keys.
__device__ __forceinline__ int32_t f8_units_end(const PrefillCursor &cur, int32_t T) {
    const int32_t keys = cur.t.p0 + 1;
    return keys <= 0 ? cur.j0 : min(cur.j1, (keys - 1) / T + 1);  // keys + T may pass 2^31
}

template <int D>
__device__ __forceinline__ void f8_producer(const PrefillArgs &a, const F8Args &f, uint8_t *smem, const CUtensorMap *tmk,
                                            const CUtensorMap *tmv, uint64_t *full, uint64_t *empty, PrefillCursor cur,
                                            int lane) {
    using L = F8Smem<D>;
    if (lane == 0) {
        prefetch_tmap(tmk);
        prefetch_tmap(tmv);
    }
    const uint64_t policy = l2_policy_evict_first();  // the codes are read once
    const uint32_t tiles = smem_u32(smem), scales = tiles + L::scales(f.stages);
    const int32_t nbox = f.T / f.gran;  // at most 16, one per lane
    const uint32_t box_bytes = (uint32_t)(f.gran * f.NH * D), sc_bytes = (uint32_t)(f.gran * f.Hk);
    uint32_t n = 0;
    bool abort = false;
    // table entry of this lane's box of unit j of a sequence (0 without that box)
    auto entry_of = [&](const PrefillTile &t, int32_t j) {
        return lane < nbox && (int64_t)j * f.T + lane * f.gran <= t.p0
                   ? a.tables[(int64_t)t.seq * a.max_blocks + (j * f.T + lane * f.gran) / a.B]
                   : 0;
    };
    int32_t phys = entry_of(cur.t, cur.j0), phys_next;
    do {
        const int32_t keys = cur.t.p0 + 1, je = f8_units_end(cur, f.T);
        auto has = [&](int32_t j) { return lane < nbox && (int64_t)j * f.T + lane * f.gran < keys; };
        auto entry = [&](int32_t j) { return entry_of(cur.t, j); };
        phys_next = entry_of(cur.t_next, 0);  // the next segment starts with its sequence
        for (int32_t j = cur.j0; j < je; ++j, ++n) {
            const uint32_t st = n % f.stages;
            const bool box = has(j), good = phys >= 0 && phys < a.NB;
            const int32_t at = good ? phys * a.B + (j * f.T + lane * f.gran) % a.B : a.NB * a.B;
            if (j + 1 < je) phys = entry(j + 1);
            if (n >= (uint32_t)f.stages && !abort && !mbar_wait_bounded(smem_u32(&empty[st]), (n / f.stages + 1) & 1)) {
                atomicOr(a.err, kErrTimeout);
                abort = true;
            }
            if (__any_sync(0xffffffffu, abort)) break;
            const uint32_t ks = scales + st * 2 * f.scale_bytes + (uint32_t)lane * sc_bytes, vs = ks + f.scale_bytes;
            if (box && !good) {  // a bad entry reads zeros: codes past the pool, the smallest scale
                atomicOr(a.err, kErrBounds);
                for (uint32_t i = 0; i < sc_bytes; i += 4) {
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(ks + i), "r"(0u) : "memory");
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(vs + i), "r"(0u) : "memory");
                }
                fence_proxy_async_smem();  // before a later copy to the same bytes
            }
            __syncwarp();  // every lane's zeros are in place before lane 0 publishes the stage
            const uint32_t boxes = (uint32_t)__popc(__ballot_sync(0xffffffffu, box));
            const uint32_t goods = (uint32_t)__popc(__ballot_sync(0xffffffffu, box && good));
            const uint32_t fb = smem_u32(&full[st]);
            if (lane == 0) mbar_arrive_expect_tx(fb, 2 * (boxes * box_bytes + goods * sc_bytes));
            __syncwarp();
            if (box) {
                const uint32_t dst = tiles + st * 2 * L::kTile + (uint32_t)lane * box_bytes;
                tma_load_3d_hint(dst, tmk, fb, 0, at, cur.kvh * f.NH, policy);
                tma_load_3d_hint(dst + L::kTile, tmv, fb, 0, at, cur.kvh * f.NH, policy);
                if (good) {
                    bulk_load(ks, a.k_scale + (int64_t)at * f.Hk, sc_bytes, fb);
                    bulk_load(vs, a.v_scale + (int64_t)at * f.Hk, sc_bytes, fb);
                }
            }
        }
        if (__any_sync(0xffffffffu, abort)) break;
        phys = phys_next;
    } while (cur.next(a));
    // copies in flight land before the CTA may exit
    bool late = false;
    for (uint32_t k = n > (uint32_t)f.stages ? n - f.stages : 0; k < n && !late; ++k)
        late = !mbar_wait_bounded(smem_u32(&full[k % f.stages]), (k / f.stages) & 1);
}

// Moves a warp's walk on: every lane works on its own copy and all store the
// same one.
__device__ __forceinline__ bool f8_next(PrefillCursor &cur, const PrefillArgs &a) {
    PrefillCursor mine = cur;
    __syncwarp();
    const bool more = mine.next(a);
    cur = mine;
    __syncwarp();
    return more;
}

template <int D>
__global__ void __launch_bounds__(kF8Threads, 2)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ PrefillArgs a, const F8Args f) {
    using L = F8Smem<D>;
    constexpr int NC = D / 16;      // 16-byte chunks of a code row
    constexpr int SH = D == 128 ? 0 : 1;  // TMA swizzle: chunk ^ (line & 7) of 128-byte lines, chunk ^ (line / 2 & 3) of 64-byte ones
    constexpr uint32_t SM = D == 128 ? 7 : 3;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *full = (uint64_t *)(smem + L::bars(f.stages, f.scale_bytes)), *empty = full + f.stages;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < f.stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), kF8Warps);
        }
        fence_mbarrier_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t c = blockIdx.x;
    // Each warp's walk, in shared memory: it is used between segments only.
    __shared__ PrefillCursor curs[kF8Warps + 1];
    PrefillCursor &cur = curs[warp];
    {
        PrefillCursor first;
        const bool work = first.init(a, c);
        if (tid == 32 * kF8Warps) note_cut(a, c, work, first);
        if (!work) return;
        cur = first;  // the same in every lane
    }
    __syncwarp();
    if (warp == kF8Warps) {
        f8_producer<D>(a, f, smem, &tmk, &tmv, full, empty, cur, lane);
        return;
    }

    const int r = lane >> 2, cq = lane & 3;  // mma group, thread in group
    const int h = warp % f.NH, sub = warp / f.NH;  // KV head of the stage, 16-token slice
    const int nsub = kF8Warps / f.NH;
    const uint32_t tiles = smem_u32(smem);
    const uint8_t *sc = smem + L::scales(f.stages);
    // ldmatrix row of this lane: token (lane & 7) + 8 (matrix & 1) of the
    // slice, chunk parity matrix >> 1
    const int mi = lane >> 3;
    const int tk = sub * 16 + (lane & 7) + (mi & 1) * 8;
    const uint32_t line = (uint32_t)(tk % f.gran);
    const uint32_t row_off = (uint32_t)(((tk / f.gran) * f.NH + h) * f.gran) * D + line * D;
    const uint32_t swz = (line >> SH) & SM;
    // chunk j + (mi >> 1), j even: (j | mi >> 1) ^ swz = j ^ (mi >> 1 ^ swz), and
    // tiles are aligned to 128 bytes
    const uint32_t lane_off = row_off + ((((uint32_t)mi >> 1) ^ swz) << 4);
    // scale bytes of token r of the slice
    const uint32_t sc_head = (uint32_t)((sub * 16 + r) * f.Hk + h);
    int st = 0;
    uint32_t phase = 0;
    bool abort = false;
    do {
        const PrefillTile t = cur.t;
        const int32_t keys = t.p0 + 1, j0 = cur.j0, je = f8_units_end(cur, f.T);
        const uint32_t sc_off = sc_head + (uint32_t)(cur.kvh * f.NH);
        const int32_t head0 = (cur.kvh * f.NH + h) * f.G;  // first query head of this warp's KV head
        // Q: column n = query head r; per 16-element chunk this thread's elements 4 cq .. + 3
        uint32_t qf[NC][2];
        float qs0, qs1;  // 2^eq scale log2(e) of this thread's columns 2 cq, 2 cq + 1
        {
            uint32_t w[NC][2];
            uint32_t am = 0;
            const uint32_t *qp = reinterpret_cast<const uint32_t *>((const __nv_bfloat16 *)a.q +
                                                                    ((int64_t)t.row0 * a.H + head0 + (r < f.G ? r : 0)) * D);
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    w[j][k] = r < f.G ? qp[8 * j + 2 * cq + k] : 0u;
                    am = max(am, max(finite_bits(__uint_as_float(w[j][k] << 16)),
                                     finite_bits(__uint_as_float(w[j][k] & 0xffff0000u))));
                }
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
            // the largest |q| to [2^14, 2^15): exponent field 141; shifts within fp32's normal range
            const int32_t eq = am == 0 ? 0 : min(max((int32_t)(am >> 23) - 141, -126), 126);
            const float mul = __uint_as_float((uint32_t)(127 - eq) << 23);
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    qf[j][k] = pack_f16x2(__uint_as_float(w[j][k] << 16) * mul,
                                          __uint_as_float(w[j][k] & 0xffff0000u) * mul);
            const float back = __uint_as_float((uint32_t)(127 + eq) << 23) * a.scale_log2;
            qs0 = __shfl_sync(0xffffffffu, back, (2 * cq) * 4);  // lane 4 n holds column n's
            qs1 = __shfl_sync(0xffffffffu, back, (2 * cq + 1) * 4);
        }
        // The next sequence's queries of this head on their way to L2 (G * D * 2
        // bytes, a line per lane).
        if (lane * 64 < f.G * D)
            asm volatile("prefetch.global.L2 [%0];" ::"l"((const __nv_bfloat16 *)a.q +
                                                          ((int64_t)cur.t_next.row0 * a.H + head0) * D + lane * 64));
        float o[NC][4];
#pragma unroll
        for (int j = 0; j < NC; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, v0 = -INFINITY, v1 = -INFINITY;  // m and m' of both columns
        float c0 = 0.f, c1 = 0.f;                                              // 2^(m - m')
        float l0 = 0.f, l1 = 0.f;
        for (int32_t j = j0; j < je; ++j) {
            if (!abort && !__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&full[st]), phase))) {
                // run on without waiting: every barrier still gets its
                // arrivals; the error word marks the output as unreliable
                if (lane == 0) atomicOr(a.err, kErrTimeout);
                abort = true;
            }
            const int32_t rest = keys - (j * f.T + sub * 16);  // tokens of this slice and after it
            if (rest > 0) {
                const uint32_t kb = tiles + (uint32_t)st * 2 * L::kTile + lane_off, vb = kb + L::kTile;
                // scale bytes of tokens r and r + 8
                const uint8_t *ks = sc + (uint32_t)st * 2 * f.scale_bytes + sc_off, *vs = ks + f.scale_bytes;
                const uint32_t ka = ks[0], kc = ks[8 * f.Hk], va = vs[0], vc = vs[8 * f.Hk];
                float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j2 = 0; j2 < NC; j2 += 2) {
                    uint32_t w[4], lo[4], hi[4];
                    ldmatrix_x4(kb ^ (uint32_t)(j2 << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) codes_f16(w[k], lo[k], hi[k]);
                    mma_f16_16816(s, lo[0], lo[1], hi[0], hi[1], qf[j2][0], qf[j2][1]);
                    mma_f16_16816(s, lo[2], lo[3], hi[2], hi[3], qf[j2 + 1][0], qf[j2 + 1][1]);
                }
                // Byte 255 is NaN, K's or V's: the row's score takes it to l and to
                // every column of O (V's own factor stays out of it, as it may
                // belong to a masked token).
                const float fa = max(ka, va) == 255u ? scale_of(255u) : scale_bits(ka);
                const float fc = max(kc, vc) == 255u ? scale_of(255u) : scale_bits(kc);
                float x0 = s[0] * (fa * qs0), x1 = s[1] * (fa * qs1);
                float x2 = s[2] * (fc * qs0), x3 = s[3] * (fc * qs1);
                if (rest < 16) {
                    if (r >= rest) x0 = x1 = -INFINITY;
                    if (r + 8 >= rest) x2 = x3 = -INFINITY;
                }
                const float ga = scale_bits(va), gc = scale_bits(vc);
                float p0, p1, p2, p3, P0, P1, P2, P3;
                auto weigh = [&]() {
                    p0 = ex2_approx(x0 - m0), p1 = ex2_approx(x1 - m1);
                    p2 = ex2_approx(x2 - m0), p3 = ex2_approx(x3 - m1);
                    // the bound keeps a factor that overflows beside p = 0 finite
                    P0 = p0 * fminf(ga * c0, kMaxFactor), P1 = p1 * fminf(ga * c1, kMaxFactor);
                    P2 = p2 * fminf(gc * c0, kMaxFactor), P3 = p3 * fminf(gc * c1, kMaxFactor);
                };
                weigh();
                // Lazy running maxima: moved only when some p or P passes
                // 2^kLazyMaxSlack times its value at the maximum (always on a
                // segment's first tokens).
                const float top = fmaxf(fmaxf(fmaxf(p0, p1), fmaxf(p2, p3)),
                                        kTopScale * fmaxf(fmaxf(P0, P1), fmaxf(P2, P3)));
                if (__any_sync(0xffffffffu, top > kTopP || m0 == -INFINITY || m1 == -INFINITY)) {
                    const float ea = (float)va - 127.f, ec = (float)vc - 127.f;
                    float a0 = fmaxf(x0, x2), a1 = fmaxf(x1, x3);
                    float b0 = fmaxf(x0 + ea, x2 + ec), b1 = fmaxf(x1 + ea, x3 + ec);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, off));
                        a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, off));
                        b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, off));
                        b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, off));
                    }
                    // a reference that stays (also at -inf) keeps its factor 1
                    if (a0 > m0) l0 *= ex2_approx(m0 - a0), m0 = a0;
                    if (a1 > m1) l1 *= ex2_approx(m1 - a1), m1 = a1;
                    // 2^(m - m') stays finite: rows of zeros have the smallest exponent
                    b0 = fmaxf(b0 - kTopBits, m0 - 126.f), b1 = fmaxf(b1 - kTopBits, m1 - 126.f);
                    const float f0 = b0 > v0 ? ex2_approx(v0 - b0) : 1.f, f1 = b1 > v1 ? ex2_approx(v1 - b1) : 1.f;
                    v0 = fmaxf(v0, b0), v1 = fmaxf(v1, b1);
                    c0 = ex2_approx(m0 - v0), c1 = ex2_approx(m1 - v1);
#pragma unroll
                    for (int jj = 0; jj < NC; ++jj) o[jj][0] *= f0, o[jj][1] *= f1, o[jj][2] *= f0, o[jj][3] *= f1;
                    weigh();
                }
                l0 += p0 + p2;
                l1 += p1 + p3;
                const uint32_t pb0 = movmatrix_trans(pack_f16x2(P0, P1));
                const uint32_t pb1 = movmatrix_trans(pack_f16x2(P2, P3));
                // Tokens past the sequence's end may hold NaN codes: zeros in
                // their place (a word holds tokens 2 cq and 2 cq + 1).
                auto add_v = [&](uint32_t keep_a, uint32_t keep_c) {
#pragma unroll
                    for (int j2 = 0; j2 < NC; j2 += 2) {
                        uint32_t w[4], lo[4], hi[4];
                        ldmatrix_x4_trans(vb ^ (uint32_t)(j2 << 4), w[0], w[1], w[2], w[3]);
                        // codes (token, column): t0d0 t0d1 t1d0 t1d1 -> t0d0 t1d0, t0d1 t1d1
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            codes_f16(__byte_perm(w[k] & (k & 1 ? keep_c : keep_a), 0u, 0x3120), lo[k], hi[k]);
                        mma_f16_16816(o[j2], lo[0], hi[0], lo[1], hi[1], pb0, pb1);
                        mma_f16_16816(o[j2 + 1], lo[2], hi[2], lo[3], hi[3], pb0, pb1);
                    }
                };
                if (rest >= 16) {
                    add_v(0xffffffffu, 0xffffffffu);
                } else {
                    const int32_t ra = rest - 2 * cq, rc = ra - 8;
                    add_v(ra >= 2 ? 0xffffffffu : ra == 1 ? 0x0000ffffu : 0u,
                          rc >= 2 ? 0xffffffffu : rc == 1 ? 0x0000ffffu : 0u);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
            if (++st == f.stages) st = 0, phase ^= 1u;
        }
        // l over the group's lanes; O in units of 2^m (in two steps: the
        // factor alone may leave fp32's range where the product does not)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, off);
            l1 += __shfl_xor_sync(0xffffffffu, l1, off);
        }
        const float g0 = v0 == -INFINITY || m0 == -INFINITY ? 0.f : ex2_approx(0.5f * (v0 - m0));
        const float g1 = v1 == -INFINITY || m1 == -INFINITY ? 0.f : ex2_approx(0.5f * (v1 - m1));
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            o[j][0] = o[j][0] * g0 * g0, o[j][2] = o[j][2] * g0 * g0;
            o[j][1] = o[j][1] * g1 * g1, o[j][3] = o[j][3] * g1 * g1;
        }
        const int h0 = 2 * cq, h1 = 2 * cq + 1;
        if (nsub > 1) {
            // Join the head's slices: warps with sub > 0 hand over (m, l) and
            // O, 64 columns at a time, and the first one folds them in order.
            float *ja = reinterpret_cast<float *>(smem + L::join(f.stages, f.scale_bytes));
            float2 *jm = reinterpret_cast<float2 *>(ja + (size_t)(kF8Warps - f.NH) * f.G * L::kJoinCols);
            auto sync = [&]() { asm volatile("bar.sync 1, %0;" ::"r"(32 * kF8Warps) : "memory"); };
            const int me = warp - f.NH;  // hand-over slot (sub > 0)
            sync();                      // the last segment's slots have been read
            if (sub > 0 && r == 0) {
                if (h0 < f.G) jm[me * f.G + h0] = make_float2(m0, l0);
                if (h1 < f.G) jm[me * f.G + h1] = make_float2(m1, l1);
            }
            sync();
            float M0 = m0, M1 = m1;
            if (sub == 0) {
                for (int q = 1; q < nsub; ++q) {
                    const int slot = (q - 1) * f.NH + h;
                    if (h0 < f.G) M0 = fmaxf(M0, jm[slot * f.G + h0].x);
                    if (h1 < f.G) M1 = fmaxf(M1, jm[slot * f.G + h1].x);
                }
                const float s0 = M0 == -INFINITY ? 0.f : ex2_approx(m0 - M0), s1 = M1 == -INFINITY ? 0.f : ex2_approx(m1 - M1);
                l0 *= s0, l1 *= s1;
#pragma unroll
                for (int j = 0; j < NC; ++j) o[j][0] *= s0, o[j][1] *= s1, o[j][2] *= s0, o[j][3] *= s1;
                for (int q = 1; q < nsub; ++q) {
                    const int slot = (q - 1) * f.NH + h;
                    if (h0 < f.G) {
                        const float2 v = jm[slot * f.G + h0];
                        l0 += M0 == -INFINITY ? v.y : v.y * ex2_approx(v.x - M0);  // (0 or NaN without a maximum)
                    }
                    if (h1 < f.G) {
                        const float2 v = jm[slot * f.G + h1];
                        l1 += M1 == -INFINITY ? v.y : v.y * ex2_approx(v.x - M1);
                    }
                }
            }
#pragma unroll
            for (int part = 0; part < D / 64; ++part) {
                if (sub > 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float *p0 = ja + ((size_t)me * f.G + h0) * L::kJoinCols + 16 * j + 2 * r, *p1 = p0 + L::kJoinCols;
                        if (h0 < f.G) *reinterpret_cast<float2 *>(p0) = make_float2(o[4 * part + j][0], o[4 * part + j][2]);
                        if (h1 < f.G) *reinterpret_cast<float2 *>(p1) = make_float2(o[4 * part + j][1], o[4 * part + j][3]);
                    }
                }
                sync();
                if (sub == 0) {
                    for (int q = 1; q < nsub; ++q) {
                        const int slot = (q - 1) * f.NH + h;
                        const float w0 = h0 < f.G && M0 != -INFINITY ? ex2_approx(jm[slot * f.G + h0].x - M0) : 0.f;
                        const float w1 = h1 < f.G && M1 != -INFINITY ? ex2_approx(jm[slot * f.G + h1].x - M1) : 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float *p0 = ja + ((size_t)slot * f.G + h0) * L::kJoinCols + 16 * j + 2 * r;
                            if (h0 < f.G) {
                                const float2 y = *reinterpret_cast<const float2 *>(p0);
                                o[4 * part + j][0] = fmaf(w0, y.x, o[4 * part + j][0]);
                                o[4 * part + j][2] = fmaf(w0, y.y, o[4 * part + j][2]);
                            }
                            if (h1 < f.G) {
                                const float2 y = *reinterpret_cast<const float2 *>(p0 + L::kJoinCols);
                                o[4 * part + j][1] = fmaf(w1, y.x, o[4 * part + j][1]);
                                o[4 * part + j][3] = fmaf(w1, y.y, o[4 * part + j][3]);
                            }
                        }
                    }
                }
                if (part + 1 < D / 64) sync();
            }
            m0 = M0, m1 = M1;
        }
        if (sub == 0) {
            if (cur.whole()) {
                const float i0 = l0 == 0.f ? 0.f : 1.f / l0, i1 = l1 == 0.f ? 0.f : 1.f / l1;
                __nv_bfloat16 *ob = (__nv_bfloat16 *)a.out + ((int64_t)t.row0 * a.H + head0) * D + 2 * r;
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    if (h0 < f.G)
                        *reinterpret_cast<uint32_t *>(ob + h0 * D + 16 * j) = pack_bf16x2(o[j][0] * i0, o[j][2] * i0);
                    if (h1 < f.G)
                        *reinterpret_cast<uint32_t *>(ob + h1 * D + 16 * j) = pack_bf16x2(o[j][1] * i1, o[j][3] * i1);
                }
            } else {
                const int64_t row = cur.slot(c) * kF8SlotRows + h * f.G;
                float *ab = a.acc + row * D + 2 * r;
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    if (h0 < f.G) *reinterpret_cast<float2 *>(ab + h0 * D + 16 * j) = make_float2(o[j][0], o[j][2]);
                    if (h1 < f.G) *reinterpret_cast<float2 *>(ab + h1 * D + 16 * j) = make_float2(o[j][1], o[j][3]);
                }
                if (r == 0) {
                    if (h0 < f.G) a.ml[row + h0] = make_float2(m0, l0);
                    if (h1 < f.G) a.ml[row + h1] = make_float2(m1, l1);
                }
            }
        }
    } while (f8_next(cur, a));
}

}  // namespace pa
