// Chunk attention on the fifth-generation tensor cores (pa_prefill for bf16,
// head_dim 64 and 128, the row layout, block sizes that are multiples of 8).
//
// A tile of the work list is two row tiles of 128 query rows (128 / G tokens x
// the G heads of one KV head, so that a K or V tile in shared memory serves
// all heads that share it); a unit is 128 keys.  Per unit and row tile
//   S[128][128] = Q K^T         D / 16 MMAs, operands in shared memory,
//   P = 2^(scale S - m)         one thread per row, P as bf16 over S's columns,
//   O[128][D] += P V            8 MMAs, P from tensor memory, V from shared.
// One CTA per SM, twelve warps: 0-3 and 4-7 are the softmax of the two row tiles
// (a thread owns one row: no shuffles), 8 issues the MMAs, 9 the TMA copies
// (10 and 11 fill up the third warpgroup).
// The two row tiles take turns on the tensor pipe: while one's S is turned
// into P, the other's O += P V and next S run.  Tensor memory holds S (128
// columns) and O (D columns) of both, 512 columns at head_dim 128.
//
// The MMAs take 4 * 128 * 128 * D FLOPs of tensor time per unit and row tile,
// the softmax 128 exponentials per row; both pipes are close to busy at
// head_dim 128, so long prompts are bound by them, and chunks of few rows over
// long contexts by the K and V bytes.
#pragma once

#include <cuda.h>  // CUtensorMap

#include "decode_merge.cuh"
#include "prefill_plan.cuh"
#include "tc_ptx.cuh"

namespace pa {

constexpr int kTcRows = 128, kTcKeys = 128, kTcThreads = 384;
// Registers: 384 threads x 168 at launch; the two softmax warpgroups take 208
// each (a row's 128 scores stay in registers), the third one keeps 88:
// 256 x 208 + 128 x 88 = 384 x 168.
constexpr int kTcSoftmaxRegs = 208, kTcOtherRegs = 88;

template <int D>
struct TcPrefill {
    static constexpr int kPanels = D / 64;
    static constexpr uint32_t kPanel = 128 * 128;            // 128 rows of 64 bf16
    static constexpr uint32_t kTile = kPanels * kPanel;      // Q row tile, K or V unit
    static constexpr int kStages = D == 128 ? 5 : 8;         // ring of K and V units
    static constexpr uint32_t kRing = 2 * kTile;             // after the two Q row tiles
    static constexpr uint32_t kBars = kRing + kStages * kTile;
    static constexpr uint32_t kBytes = kBars + 256 + 3 * D * 4;  // barriers; columns with odd values
    static constexpr size_t kSmem = kBytes + 1024;           // the base is aligned to 1024
    static constexpr uint32_t kS = 0, kO = 256;              // tensor-memory columns: S0, S1, O0, O1
};

// Barriers of a CTA, in shared memory.
struct TcBars {
    uint32_t q_full, q_free, kv_full, kv_free, s_full, p_full, o_full, o_free;  // addresses; arrays 8 bytes apart
    __device__ __forceinline__ TcBars(uint32_t base, int stages) {
        q_full = base;
        q_free = base + 8;
        s_full = base + 16;
        p_full = base + 32;
        o_full = base + 48;
        o_free = base + 64;
        kv_full = base + 80;
        kv_free = kv_full + 8 * (uint32_t)stages;
    }
};

// A bounded wait that stays off once one ran out: the roles then run through
// their loops without waiting, so that every barrier still gets its arrivals
// and the CTA ends; the error word marks the call's output as unreliable.
__device__ __forceinline__ void tc_wait(uint32_t bar, uint32_t parity, bool &abort, unsigned int *err) {
    if (abort) return;
    if (!mbar_wait_bounded(bar, parity)) {
        atomicOr(err, kErrTimeout);
        abort = true;
    }
}

// Units of a segment that each row tile takes: [j0, je[i]).
struct TcSegment {
    PrefillTile t;
    int32_t keys;   // keys the tile sees
    int32_t je[2], jend;
    __device__ __forceinline__ TcSegment(const PrefillArgs &a, const PrefillCursor &cur) {
        t = a.tiles[cur.k];
        keys = t.p0 + t.ntok;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int32_t n = min(t.ntok, (i + 1) * a.tq1);  // tokens up to this row tile's end
            const int32_t ki = t.ntok > i * a.tq1 ? max(t.p0 + n, 0) : 0;
            je[i] = min(cur.j1, (ki + kTcKeys - 1) / kTcKeys);
        }
        jend = max(je[0], je[1]);
    }
};

// ------------------------------------------------------------ TMA producer
// One warp.  Per segment the Q rows (one box of tq1 tokens x G heads per row
// tile and 64-element panel), then K and V units through the ring, K first.
// A unit is 128 / gran boxes per panel, gran = gcd(block size, 128) keys, one
// box per lane; the block-table entries of a unit are read one unit ahead.
template <int D>
__device__ __forceinline__ void tc_producer(const PrefillArgs &a, uint8_t *smem, const TcBars &bar,
                                            const CUtensorMap *tmq, const CUtensorMap *tmk, const CUtensorMap *tmv,
                                            int32_t gran, PrefillCursor cur, int lane) {
    using L = TcPrefill<D>;
    if (lane == 0) {
        prefetch_tmap(tmq);
        prefetch_tmap(tmk);
        prefetch_tmap(tmv);
    }
    const uint32_t q_dst = smem_u32(smem), ring = q_dst + L::kRing;
    const int32_t nbm = kTcKeys / gran;  // boxes of a unit per panel (at most 16)
    const int32_t bi = lane % nbm, panel = lane / nbm;
    const bool has_box = panel < L::kPanels;
    const uint32_t box_off = (uint32_t)panel * L::kPanel + (uint32_t)(bi * gran) * 128u;
    uint32_t n = 0, segs = 0;  // ring entries and Q loads issued
    bool abort = false;
    do {
        const TcSegment sg(a, cur);
        if (sg.jend <= cur.j0) continue;
        const int32_t *row = a.tables + (int64_t)sg.t.seq * a.max_blocks;
        auto entry = [&](int32_t j) -> int32_t {  // pool row of this lane's box of unit j, -1: no box
            const int64_t pos = (int64_t)j * kTcKeys + bi * gran;
            if (!has_box || pos >= sg.keys) return -1;
            const int32_t p = (int32_t)pos, blk = p / a.B, phys = row[blk];
            if (phys < 0 || phys >= a.NB) {  // reads zeros: the box lies past the pool
                atomicOr(a.err, kErrBounds);
                return a.NB * a.B;
            }
            return phys * a.B + (p - blk * a.B);
        };
        int32_t next = entry(cur.j0);
        if (segs > 0) tc_wait(bar.q_free, (segs - 1) & 1, abort, a.err);
        if (__any_sync(0xffffffffu, abort)) break;
        if (lane == 0) {
            const int32_t nrt = sg.t.ntok > a.tq1 ? 2 : 1;
            mbar_arrive_expect_tx(bar.q_full, (uint32_t)(nrt * L::kPanels * a.tq1 * a.G) * 128u);
            for (int32_t i = 0; i < nrt; ++i)
                for (int32_t p = 0; p < L::kPanels; ++p)
                    tma_load_4d(q_dst + i * L::kTile + p * L::kPanel, tmq, bar.q_full, 0, p, cur.kvh * a.G,
                                sg.t.row0 + i * a.tq1);
        }
        ++segs;
        for (int32_t j = cur.j0; j < sg.jend; ++j) {
            const int32_t at = next;
            if (j + 1 < sg.jend) next = entry(j + 1);
            const uint32_t bytes =
                (uint32_t)__popc(__ballot_sync(0xffffffffu, at >= 0)) * (uint32_t)gran * 128u;  // of K, and of V
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++n) {
                const uint32_t st = n % L::kStages;
                if (n >= L::kStages) tc_wait(bar.kv_free + 8 * st, (n / L::kStages + 1) & 1, abort, a.err);
                if (__any_sync(0xffffffffu, abort)) break;
                if (lane == 0) mbar_arrive_expect_tx(bar.kv_full + 8 * st, bytes);
                __syncwarp();
                if (at >= 0)
                    tma_load_4d(ring + st * L::kTile + box_off, kv == 0 ? tmk : tmv, bar.kv_full + 8 * st, 0, at, panel,
                                cur.kvh);
            }
            if (__any_sync(0xffffffffu, abort)) break;
        }
        if (__any_sync(0xffffffffu, abort)) break;
    } while (cur.next(a));
    // Copies in flight, and the issuer's last arrivals on the free barriers,
    // land before the CTA may exit.
    bool late = false;
    for (uint32_t k = n > (uint32_t)L::kStages ? n - L::kStages : 0; k < n; ++k) {
        tc_wait(bar.kv_full + 8 * (k % L::kStages), (k / L::kStages) & 1, late, a.err);
        tc_wait(bar.kv_free + 8 * (k % L::kStages), (k / L::kStages) & 1, late, a.err);
    }
    if (segs > 0) {
        tc_wait(bar.q_full, (segs - 1) & 1, late, a.err);
        tc_wait(bar.q_free, (segs - 1) & 1, late, a.err);
    }
}

// Columns of V with values that are not finite at keys that only some rows of
// a tile see (the tile's own tokens): 0 x V is not 0 there, so such a value is
// replaced by 0 before the products, and each column keeps the first
// position that holds +inf, -inf and NaN; rows that see it add it at the end.
struct OddColumns {
    int32_t *first;  // [3][D]: +inf, -inf, NaN; kNone without one
    static constexpr int32_t kNone = 0x7fffffff;
};

// Rows [r0, r1) of a staged V unit: values that are not finite to
// odd.first, zeros in their place; rows [r1, r2) all zeros.  One warp.
// Returns whether any was found.
template <int D>
__device__ __forceinline__ bool tc_clean_v(uint32_t vbase, int r0, int r1, int r2, int32_t pos0, const OddColumns &odd,
                                           int lane) {
    using L = TcPrefill<D>;
    bool found = false;
    constexpr int kChunks = D / 8;  // 16-byte chunks of a row
    for (int e = r0 * kChunks + lane; e < r2 * kChunks; e += 32) {
        const int r = e / kChunks, ch = e % kChunks;
        const uint32_t addr =
            vbase + (uint32_t)(ch >> 3) * L::kPanel + (uint32_t)r * 128u + (uint32_t)(((ch & 7) ^ (r & 7)) << 4);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        bool store = r >= r1;
        if (!store) {
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(addr));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t h = (w[k >> 1] >> (16 * (k & 1))) & 0xffffu;
                if ((h & 0x7f80u) == 0x7f80u) {
                    const int kind = (h & 0x7fu) ? 2 : (h >> 15);
                    atomicMin(&odd.first[kind * D + ch * 8 + k], pos0 + r);
                    w[k >> 1] &= k & 1 ? 0x0000ffffu : 0xffff0000u;
                    store = found = true;
                }
            }
        }
        if (store)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
    }
    fence_proxy_async_smem();  // the MMAs read these rows through the async proxy
    return __any_sync(0xffffffffu, found);
}

// -------------------------------------------------------------- MMA issuer
// One warp; lane 0 issues.  MMAs of one thread complete in order, so S of a
// unit may be computed over the P of the one before (its O += P V was issued
// earlier), and a row tile's S being complete says that its earlier O is too.
template <int D>
__device__ __forceinline__ void tc_issuer(const PrefillArgs &a, uint8_t *smem, const TcBars &bar, uint32_t tmem,
                                          const OddColumns &odd, int32_t *odd_flag, PrefillCursor cur, int lane) {
    using L = TcPrefill<D>;
    constexpr uint32_t IDESC_S = tc_idesc_bf16(128, kTcKeys, false, false);
    constexpr uint32_t IDESC_O = tc_idesc_bf16(128, D, false, true);
    const uint32_t q_base = smem_u32(smem), ring = q_base + L::kRing;
    uint32_t n = 0, segs = 0;        // ring entries consumed, segments
    uint32_t np[2] = {0, 0};         // P tiles taken per row tile
    uint32_t no[2] = {0, 0};         // segments with units per row tile
    bool abort = false, odd_dirty = false;
    do {
        const TcSegment sg(a, cur);
        if (sg.jend <= cur.j0) continue;
        tc_wait(bar.q_full, segs & 1, abort, a.err);
        ++segs;
        // The row tile's earlier rows have left O and the odd columns.  Waited
        // for once per segment: a row tile may finish this segment (and
        // complete the barrier's next phase) units before the other does.
        bool rows_read[2] = {no[0] == 0, no[1] == 0};
        auto wait_rows_read = [&](int i) {
            if (!rows_read[i]) tc_wait(bar.o_free + 8 * i, (no[i] - 1) & 1, abort, a.err);
            rows_read[i] = true;
        };
        auto issue_s = [&](int i, uint32_t kbase) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (uint32_t)(k >> 2) * L::kPanel + (uint32_t)(k & 3) * 32;
                tc_mma_bf16(tmem + L::kS + i * 128, smem_desc_sw128(q_base + i * L::kTile + off, 16, 1024),
                            smem_desc_sw128(kbase + off, 16, 1024), IDESC_S, k > 0 ? 1u : 0u);
            }
            tc_commit(bar.s_full + 8 * i);
        };
        uint32_t st = n % L::kStages;
        tc_wait(bar.kv_full + 8 * st, (n / L::kStages) & 1, abort, a.err);
        ++n;
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (cur.j0 < sg.je[i]) issue_s(i, ring + st * L::kTile);
            tc_commit(bar.kv_free + 8 * st);
            if (cur.j0 + 1 == sg.jend) tc_commit(bar.q_free);
        }
        __syncwarp();
        for (int32_t j = cur.j0; j < sg.jend; ++j) {
            const uint32_t sv = n % L::kStages;
            const uint32_t vbase = ring + sv * L::kTile;
            tc_wait(bar.kv_full + 8 * sv, (n / L::kStages) & 1, abort, a.err);
            ++n;
            // keys of this unit that not every row sees, or that no row does
            const int32_t pos0 = j * kTcKeys;
            const int nk = min(kTcKeys, sg.keys - pos0), nk16 = (nk + 15) & ~15;
            const int shared = min(nk, max(0, sg.t.p0 + 1 - pos0));
            if (shared < nk16) {
                wait_rows_read(0);
                wait_rows_read(1);
                if (odd_dirty) {  // an earlier tile's columns
                    for (int e = lane; e < 3 * D; e += 32) odd.first[e] = OddColumns::kNone;
                    if (lane == 0) *odd_flag = 0;
                    odd_dirty = false;
                    __syncwarp();
                }
                if (tc_clean_v<D>(vbase, shared, nk, nk16, pos0, odd, lane)) {
                    if (lane == 0) *odd_flag = 1;
                }
                __syncwarp();
            }
            const bool more = j + 1 < sg.jend;
            const uint32_t sk = n % L::kStages;
            const uint32_t nk_par = (n / L::kStages) & 1;
            if (more) ++n;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (j < sg.je[i]) {
                    if (j == cur.j0) {  // O is about to be overwritten
                        wait_rows_read(i);
                        ++no[i];
                    }
                    tc_wait(bar.p_full + 8 * i, np[i] & 1, abort, a.err);
                    ++np[i];
                    tc_fence_after();
                    if (lane == 0) {
                        for (int k = 0; k < nk16 / 16; ++k)
                            tc_mma_bf16_ta(tmem + L::kO + i * D, tmem + L::kS + i * 128 + k * 8,
                                           smem_desc_sw128(vbase + (uint32_t)k * 2048, L::kPanel, 1024), IDESC_O,
                                           j > cur.j0 || k > 0 ? 1u : 0u);
                        if (j + 1 == sg.je[i]) tc_commit(bar.o_full + 8 * i);
                    }
                    __syncwarp();
                }
                if (more && i == 0) tc_wait(bar.kv_full + 8 * sk, nk_par, abort, a.err);
                if (j + 1 < sg.je[i]) {
                    tc_fence_after();
                    if (lane == 0) issue_s(i, ring + sk * L::kTile);
                    __syncwarp();
                }
            }
            if (lane == 0) {
                tc_commit(bar.kv_free + 8 * sv);
                if (more) tc_commit(bar.kv_free + 8 * sk);
                if (j + 2 == sg.jend) tc_commit(bar.q_free);
            }
            __syncwarp();
        }
        odd_dirty = *odd_flag != 0;  // written by this warp alone
    } while (cur.next(a));
    // Every MMA ends in an o_full that the softmax warps wait for; nothing of
    // this warp is in flight once they have (see the kernel's end).
}

// ----------------------------------------------------------------- softmax
// Four warps per row tile; a thread owns one query row (tensor-memory lane).
template <int D>
__device__ __forceinline__ void tc_softmax(const PrefillArgs &a, const TcBars &bar, uint32_t tmem,
                                           const OddColumns &odd, const int32_t *odd_flag, PrefillCursor cur, int32_t c,
                                           int i, int warp, int lane) {
    using L = TcPrefill<D>;
    const int r = warp * 32 + lane;  // row of the row tile
    const uint32_t t_lane = (uint32_t)(warp * 32) << 16;
    const uint32_t tS = tmem + L::kS + i * 128 + t_lane, tO = tmem + L::kO + i * D + t_lane;
    const uint32_t s_full = bar.s_full + 8 * i, p_full = bar.p_full + 8 * i;
    const int tok_r = r / a.G, g = r - tok_r * a.G;
    const float sl = a.scale_log2;
    uint32_t ns = 0, no = 0;
    bool abort = false;
    do {
        const TcSegment sg(a, cur);
        const int32_t tok = i * a.tq1 + tok_r;
        const bool valid = tok_r < a.tq1 && tok < sg.t.ntok;
        const bool warp_rows = __any_sync(0xffffffffu, valid);
        const int32_t last = sg.t.p0 + tok;
        const int32_t je = sg.je[i];
        float m = -INFINITY, l = 0.f;
        for (int32_t j = cur.j0; j < je; ++j) {
            tc_wait(s_full, ns & 1, abort, a.err);
            ++ns;
            tc_fence_after();
            if (warp_rows) {
                float x[128];
                tmem_ld128(tS, x);
                const int32_t nvis = last - j * kTcKeys + 1;
                if (__any_sync(0xffffffffu, valid && nvis < kTcKeys)) {
#pragma unroll
                    for (int k = 0; k < 128; ++k) x[k] = k < nvis ? x[k] : -INFINITY;
                }
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int k = 4; k < 128; k += 8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mx[q] = k + q + 4 < 128 ? fmaxf(fmaxf(mx[q], x[k + q]), x[k + q + 4]) : fmaxf(mx[q], x[k + q]);
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
                // Lazy running maximum: moved (with l and O rescaled) only when
                // a score passes it by more than kLazyMaxSlack.
                const bool grow = valid && top > m + kLazyMaxSlack;
                if (__any_sync(0xffffffffu, grow)) {
                    const float mn = grow ? top : m;
                    const float al = grow ? ex2_approx(m - mn) : 1.f;
                    m = mn;
                    l *= al;
                    if (j > cur.j0) {
#pragma unroll 1
                        for (int d0 = 0; d0 < D; d0 += 32) {
                            float o[32];
                            tmem_ld32(tO + (uint32_t)d0, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= al;
                            tmem_st32(tO + (uint32_t)d0, o);
                        }
                    }
                }
                const float mref = m == -INFINITY ? 0.f : m;  // a row without keys so far: zeros
                const uint64_t sl2 = f32x2(sl, sl), mm2 = f32x2(-mref, -mref);
                uint64_t sum[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        float y0, y1;
                        f32x2_get(fma_f32x2(f32x2(x[64 * h + 2 * k], x[64 * h + 2 * k + 1]), sl2, mm2), y0, y1);
                        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                        sum[k & 1] = add_f32x2(sum[k & 1], f32x2(p0, p1));
                        w[k] = pack_bf16x2(p0, p1);
                    }
                    tmem_st32_async(tS + 32 * h, w);
                }
                float s0, s1;
                f32x2_get(add_f32x2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
        }
        const bool any = je > cur.j0;
        if (any) {
            tc_wait(bar.o_full + 8 * i, no & 1, abort, a.err);
            ++no;
            tc_fence_after();
        }
        const bool whole = cur.whole();
        const int64_t row = cur.slot(c) * (2 * kTcRows) + i * kTcRows + r;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool odd_tile = any && *odd_flag != 0;
        __nv_bfloat16 *op =
            (__nv_bfloat16 *)a.out + ((int64_t)(sg.t.row0 + tok) * a.H + (int64_t)cur.kvh * a.G + g) * D;
        if (warp_rows) {
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
                float o[32];
                if (any) {
                    tmem_ld32(tO + (uint32_t)d0, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0.f;
                }
                if (odd_tile) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (last >= odd.first[d0 + k]) o[k] += INFINITY;
                        if (last >= odd.first[D + d0 + k]) o[k] -= INFINITY;
                        if (last >= odd.first[2 * D + d0 + k]) o[k] += __uint_as_float(0x7fffffffu);
                    }
                }
                if (valid) {
                    if (whole) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
                            *reinterpret_cast<uint4 *>(op + d0 + k) =
                                make_uint4(pack_bf16x2(o[k] * inv, o[k + 1] * inv),
                                           pack_bf16x2(o[k + 2] * inv, o[k + 3] * inv),
                                           pack_bf16x2(o[k + 4] * inv, o[k + 5] * inv),
                                           pack_bf16x2(o[k + 6] * inv, o[k + 7] * inv));
                    } else {
                        float *ap = a.acc + row * D + d0;
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4 *>(ap + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    }
                }
            }
            if (valid && !whole) a.ml[row] = make_float2(m, l);
        }
        if (any) {  // O (and the odd columns) have been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.o_free + 8 * i);
        }
    } while (cur.next(a));
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const PrefillArgs a, const int32_t gran) {
    using L = TcPrefill<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const TcBars bar(smem_u32(smem + L::kBars), L::kStages);
    uint32_t *tmem_slot = (uint32_t *)(smem + L::kBars + 248);
    int32_t *odd_flag = (int32_t *)(smem + L::kBars + 252);
    OddColumns odd{(int32_t *)(smem + L::kBars + 256)};
    static_assert(80 + 16 * L::kStages <= 248, "the barriers fit");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(bar.q_full, 1);
        mbar_init(bar.q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar.s_full + 8 * i, 1);
            mbar_init(bar.p_full + 8 * i, 4);
            mbar_init(bar.o_full + 8 * i, 1);
            mbar_init(bar.o_free + 8 * i, 4);
        }
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar.kv_full + 8 * s, 1);
            mbar_init(bar.kv_free + 8 * s, 1);
        }
        *odd_flag = 0;
        fence_mbarrier_init();
    }
    for (int e = tid; e < 3 * D; e += kTcThreads) odd.first[e] = OddColumns::kNone;
    if (warp == 8) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t c = blockIdx.x;
    PrefillCursor cur;
    if (cur.init(a, c)) {
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcSoftmaxRegs));
            tc_softmax<D>(a, bar, tmem, odd, odd_flag, cur, c, warp >> 2, warp & 3, lane);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcOtherRegs));
            if (warp == 8)
                tc_issuer<D>(a, smem, bar, tmem, odd, odd_flag, cur, lane);
            else if (warp == 9)
                tc_producer<D>(a, smem, bar, &tmq, &tmk, &tmv, gran, cur, lane);
        }
    }
    // The softmax warps have waited for the last o_full, which every MMA
    // precedes: nothing uses the tensor memory any more.
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace pa
