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
// (a thread owns one row: no shuffles), 8 issues the MMAs, 9 and 10 the
// TMA copies, 11 guards V's masked rows.
// The two row tiles take turns on the tensor pipe: while one's S is turned
// into P, the other's O += P V and next S run.  Tensor memory holds S (128
// columns) and O (D columns) of both, 512 columns at head_dim 128.
//
// P is bf16 because kind::f16 takes both operands of one type and V is bf16: an
// error of at most 2^-8 of each key's share (measured over whole outputs
// 0.0020 to 0.0024 against 64 bits, 0.0015 to 0.0017 of it the output's own rounding).
// fp16 would round finer but needs V converted, and its range; fp32 P is the
// CUDA-core kernel's.  The maximum, the sum and O are fp32, and the sum is of the
// probabilities before they are rounded.
//
// The MMAs take 4 * 128 * 128 * D FLOPs of tensor time per unit and row tile,
// the softmax 128 exponentials per row; both pipes are close to busy at
// head_dim 128, so long prompts are bound by them, and chunks of few rows over
// long contexts by the K and V bytes.  Measured, whole calls repeated on one set
// of inputs (32 / 8 heads, head_dim 128; boxes and clocks differ): a prompt of 8192
// tokens 356 to 363 us (1515 to 1546 TFLOP/s), 2048 tokens behind 30720 624 to 678
// us (1571 to 1706), 5 tokens of 64 sequences over 4096 176 to 181 us (5.9 to 6.1
// TB/s).  With three sets of inputs in turn that prompt takes 387 to 389 us (1413
// to 1419).  The extra weight of a tile, 1 / 2 / 3 / 4 units: 412 / 380 / 361 /
// 365 us on that prompt, no difference on long contexts.
#pragma once

#include <cuda.h>  // CUtensorMap

#include "decode_merge.cuh"
#include "prefill_plan.cuh"
#include "tc_ptx.cuh"

namespace pa {

constexpr int kTcRows = 128, kTcKeys = 128, kTcThreads = 384, kTcExtra = 3;
constexpr unsigned long long kTcUnitNs = 4096;
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
    uint32_t q_full, q_free, v_go, v_ok, kv_full, kv_free, s_full, p_full, o_full, o_free;  // addresses; arrays 8 bytes apart
    __device__ __forceinline__ TcBars(uint32_t base, int stages) {
        q_full = base;
        q_free = base + 8;
        s_full = base + 16;
        p_full = base + 32;
        o_full = base + 48;
        o_free = base + 64;
        v_go = base + 80;
        v_ok = base + 88;
        kv_full = base + 96;
        kv_free = kv_full + 8 * (uint32_t)stages;
    }
};

// A bounded wait that stays off once one ran out: the roles then run through
// their loops without waiting, so that every barrier still gets its arrivals
// and the CTA ends; the error word marks the call's output as unreliable.
__device__ __forceinline__ void tc_wait(uint32_t bar, uint32_t parity, bool &abort, unsigned int *err,
                                        unsigned long long limit_ns = kWaitLimitNs) {
    if (abort) return;
    if (!mbar_wait_bounded(bar, parity, limit_ns)) {
        atomicOr(err, kErrTimeout);
        abort = true;
    }
}

// Units of a segment that each row tile takes: [j0, je[i]).
struct TcSegment {
    PrefillTile t;
    int32_t keys;   // keys the tile sees
    int32_t je[2], jend;
    template <class Walk>
    __device__ __forceinline__ TcSegment(const PrefillArgs &a, const Walk &cur) {
        t = cur.t;
        keys = t.p0 + t.ntok;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int32_t n = min(t.ntok, (i + 1) * a.tq1);  // tokens up to this row tile's end
            const int32_t ki = t.ntok > i * a.tq1 ? max(t.p0 + n, 0) : 0;
            je[i] = min(cur.j1, (int32_t)(((uint32_t)ki + kTcKeys - 1) / kTcKeys));  // the sum may pass 2^31
        }
        jend = max(je[0], je[1]);
    }
};

// ----------------------------------------------------------- TMA producers
// One warp for K (and the Q rows), one for V.  Entry n of the ring is K of a
// unit for even n, V for odd n.  A unit is 128 / gran boxes per panel, gran =
// gcd(block size, 128) keys, one box per lane; the block-table entry of a
// lane's next box is read a unit ahead and looked at when its unit comes, so
// no load is waited for.  Q: one box of tq1 tokens x G heads per row tile and
// 64-element panel.
template <int D, bool kIsV>
__device__ __forceinline__ void tc_producer(const PrefillArgs &a, uint8_t *smem, const TcBars &bar,
                                            const CUtensorMap *tmq, const CUtensorMap *tm, int32_t gran,
                                            int32_t c, int lane) {
    using L = TcPrefill<D>;
    if (lane == 0) {
        if (!kIsV) prefetch_tmap(tmq);
        prefetch_tmap(tm);
    }
    const uint32_t q_dst = smem_u32(smem), ring = q_dst + L::kRing;
    const int32_t nbm = kTcKeys / gran;  // boxes of a unit per panel (at most 16)
    const int32_t bi = lane % nbm, panel = lane / nbm;
    const bool has_box = panel < L::kPanels;
    const uint32_t box_off = (uint32_t)panel * L::kPanel + (uint32_t)(bi * gran) * 128u;
    uint32_t n = kIsV ? 1 : 0, segs = 0;  // next ring entry, segments with units
    bool abort = false;
    PrefillCursor cur;
    if (!cur.init(a, c)) return;
    do {
        const TcSegment sg(a, cur);
        if (sg.jend <= cur.j0) continue;
        const int32_t *row = a.tables + (int64_t)sg.t.seq * a.max_blocks;
        auto has_key = [&](int32_t j) { return has_box && (int64_t)j * kTcKeys + bi * gran < sg.keys; };
        auto entry = [&](int32_t j) { return has_key(j) ? row[(j * kTcKeys + bi * gran) / a.B] : 0; };
        int32_t phys = entry(cur.j0);
        if (!kIsV) {
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
        }
        ++segs;
        for (int32_t j = cur.j0; j < sg.jend; ++j, n += 2) {
            const int32_t p = j * kTcKeys + bi * gran;
            const bool box = has_key(j);
            int32_t at = a.NB * a.B;  // a bad entry reads zeros: the box lies past the pool
            if (phys >= 0 && phys < a.NB)
                at = phys * a.B + p % a.B;
            else if (box)
                atomicOr(a.err, kErrBounds);
            if (j + 1 < sg.jend) phys = entry(j + 1);
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, box)) * (uint32_t)gran * 128u;
            const uint32_t st = n % L::kStages;
            if (n >= L::kStages) tc_wait(bar.kv_free + 8 * st, (n / L::kStages + 1) & 1, abort, a.err);
            if (__any_sync(0xffffffffu, abort)) break;
            if (lane == 0) mbar_arrive_expect_tx(bar.kv_full + 8 * st, bytes);
            __syncwarp();
            if (box)
                tma_load_4d(ring + st * L::kTile + box_off, tm, bar.kv_full + 8 * st, 0, at, panel, cur.kvh);
        }
        if (__any_sync(0xffffffffu, abort)) break;
    } while (cur.next(a));
    // This warp's copies in flight, and the issuer's last arrivals on the free
    // barriers, land before the CTA may exit.
    bool late = false;
    const uint32_t total = n - (kIsV ? 1u : 0u);  // ring entries of the CTA; the last kStages are not reused
    uint32_t k = total > (uint32_t)L::kStages ? total - L::kStages : 0;
    if ((k & 1u) != (kIsV ? 1u : 0u)) ++k;
    for (; k < total; k += 2) {
        tc_wait(bar.kv_full + 8 * (k % L::kStages), (k / L::kStages) & 1, late, a.err);
        tc_wait(bar.kv_free + 8 * (k % L::kStages), (k / L::kStages) & 1, late, a.err);
    }
    if (!kIsV && segs > 0) {
        tc_wait(bar.q_full, (segs - 1) & 1, late, a.err);
        tc_wait(bar.q_free, (segs - 1) & 1, late, a.err);
    }
}

// --------------------------------------------------------------- V's guard
// 0 x V is not 0 where V is not finite, and the products run over whole units:
// keys that only some rows of a tile see (its own tokens, from position
// p0 + 1 on) and the rest of the last 16 keys.  One warp looks at those rows
// of V before their products: rows past the tile's keys become zeros, and a
// value that is not finite is replaced by 0 while its column keeps the first
// position that holds +inf, -inf and NaN; the rows that see it add it at the
// end.  odd.segment names, per row tile, the last segment with such a value in
// the row tile's own units.  Its word is written before the product that ends
// those units, so the row tile's wait for its O orders the two; units that only
// the other row tile takes touch neither the word nor a position that its rows
// see, whichever moment they read the columns at.
struct OddColumns {
    int32_t *first;    // [3][D]: +inf, -inf, NaN; kNone without one
    int32_t *segment;  // [2] 1-based count of segments with units; 0: none so far
    static constexpr int32_t kNone = 0x7fffffff;
};

// First unit of a segment that holds keys for the guard.
__device__ __forceinline__ int32_t guard_from(const TcSegment &sg) { return max(sg.t.p0 + 1, 0) / kTcKeys; }

template <int D>
__device__ __forceinline__ uint32_t v_chunk(uint32_t vbase, int e) {  // address of 16-byte chunk e % (D / 8) of row e / (D / 8)
    constexpr int kChunks = D / 8;
    const int r = e / kChunks, ch = e % kChunks;
    return vbase + (uint32_t)(ch >> 3) * TcPrefill<D>::kPanel + (uint32_t)r * 128u +
           (uint32_t)(((ch & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Sign bits of the halves whose exponent is all ones (bf16 infinities and NaN).
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

template <int D>
__device__ __forceinline__ void tc_guard(const PrefillArgs &a, uint8_t *smem, const TcBars &bar, const OddColumns &odd,
                                         int32_t c, int lane) {
    using L = TcPrefill<D>;
    constexpr int kChunks = D / 8;
    const uint32_t ring = smem_u32(smem) + L::kRing;
    uint32_t n = 1, segs = 0, units = 0;  // ring entry of V, segments, guarded units
    uint32_t no[2] = {0, 0};              // earlier segments with units per row tile
    uint32_t held = 0;                    // the segment that the columns belong to
    bool abort = false;
    PrefillCursor cur;
    const bool work = cur.init(a, c);
    if (lane == 0) note_cut(a, c, work, cur);
    if (!work) return;
    do {
        const TcSegment sg(a, cur);
        if (sg.jend <= cur.j0) continue;
        ++segs;
        for (int32_t j = max(cur.j0, guard_from(sg)); j < sg.jend; ++j, ++units) {
            // The issuer has seen V arrive.  This wait and the softmax's for S
            // may last while the other roles work through most of the CTA's
            // range, so their limit grows with the range.
            tc_wait(bar.v_go, units & 1, abort, a.err, a.wait_ns);
            const uint32_t vbase = ring + ((n + 2 * (uint32_t)(j - cur.j0)) % L::kStages) * L::kTile;
            const int32_t pos0 = j * kTcKeys;
            const int nk = min(kTcKeys, sg.keys - pos0), nk16 = (nk + 15) & ~15;
            const int r0 = min(nk, max(0, sg.t.p0 + 1 - pos0));
            for (int e = nk * kChunks + lane; e < nk16 * kChunks; e += 32)
                sts128(v_chunk<D>(vbase, e), make_uint4(0u, 0u, 0u, 0u));
            uint32_t any = 0;
            int e = r0 * kChunks + lane;
            for (; e + 96 < nk * kChunks; e += 128) {  // four loads in flight
                uint4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] = lds128(v_chunk<D>(vbase, e + 32 * u));
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    any |= odd_bits(v[u].x) | odd_bits(v[u].y) | odd_bits(v[u].z) | odd_bits(v[u].w);
            }
            for (; e < nk * kChunks; e += 32) {
                const uint4 v = lds128(v_chunk<D>(vbase, e));
                any |= odd_bits(v.x) | odd_bits(v.y) | odd_bits(v.z) | odd_bits(v.w);
            }
            if (__any_sync(0xffffffffu, any != 0)) {
                // The columns are read by the rows of the segment before: wait
                // until they are through.  A row tile that began its units at
                // j0 has been waited for there (its barrier may be a phase on).
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (no[i] > 0 && (j == cur.j0 || sg.je[i] <= cur.j0))
                        tc_wait(bar.o_free + 8 * i, (no[i] - 1) & 1, abort, a.err);
                if (held != 0 && held != segs)
                    for (int x = lane; x < 3 * D; x += 32) odd.first[x] = OddColumns::kNone;
                __syncwarp();
                for (e = r0 * kChunks + lane; e < nk * kChunks; e += 32) {
                    const uint32_t addr = v_chunk<D>(vbase, e);
                    const uint4 v = lds128(addr);
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    if (!(odd_bits(v.x) | odd_bits(v.y) | odd_bits(v.z) | odd_bits(v.w))) continue;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t h = (w[k >> 1] >> (16 * (k & 1))) & 0xffffu;
                        if ((h & 0x7f80u) == 0x7f80u) {
                            const int kind = (h & 0x7fu) ? 2 : (int)(h >> 15);
                            atomicMin(&odd.first[kind * D + (e % kChunks) * 8 + k], pos0 + e / kChunks);
                            w[k >> 1] &= k & 1 ? 0x0000ffffu : 0xffff0000u;
                        }
                    }
                    sts128(addr, make_uint4(w[0], w[1], w[2], w[3]));
                }
                held = segs;
                __syncwarp();
                if (lane == 0 && j < sg.je[0]) odd.segment[0] = (int32_t)segs;
                if (lane == 1 && j < sg.je[1]) odd.segment[1] = (int32_t)segs;
            }
            fence_proxy_async_smem();  // the MMAs read these rows through the async proxy
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.v_ok);
        }
        n += 2 * (uint32_t)(sg.jend - cur.j0);
#pragma unroll
        for (int i = 0; i < 2; ++i) no[i] += cur.j0 < sg.je[i] ? 1 : 0;
    } while (cur.next(a));
}

// A value that is the same in every lane, as the compiler can see: loops and
// branches on it keep the warp converged and its descriptors in uniform
// registers.
__device__ __forceinline__ int32_t uniform(int32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// -------------------------------------------------------------- MMA issuer
// One warp; one elected lane issues.  MMAs of one thread complete in order, so S of a
// unit may be computed over the P of the one before (its O += P V was issued
// earlier), and a row tile's S being complete says that its earlier O is too.
template <int D>
__device__ __forceinline__ void tc_issuer(const PrefillArgs &a, uint8_t *smem, const TcBars &bar, uint32_t tmem,
                                          int32_t c, int lane) {
    using L = TcPrefill<D>;
    constexpr uint32_t IDESC_S = tc_idesc_bf16(128, kTcKeys, false, false);
    constexpr uint32_t IDESC_O = tc_idesc_bf16(128, D, false, true);
    const uint32_t ring = smem_u32(smem) + L::kRing;
    // Descriptors of the first Q row tile and ring entry; the others' start
    // addresses (in 16-byte units, the low bits of a descriptor) are added.
    const uint64_t q_desc = smem_desc_sw128(smem_u32(smem), 16, 1024), k_desc = smem_desc_sw128(ring, 16, 1024),
                   v_desc = smem_desc_sw128(ring, L::kPanel, 1024);
    const uint32_t one = elect_one();
    uint32_t n = 0, segs = 0, units = 0;  // ring entries consumed, segments, guarded units
    uint32_t np[2] = {0, 0};              // P tiles taken per row tile
    uint32_t no[2] = {0, 0};              // segments with units per row tile
    bool abort = false;
    PrefillCursor cur;
    if (!cur.init(a, c)) return;
    do {
        const TcSegment sg(a, cur);
        const int32_t j0 = uniform(cur.j0), jend = uniform(sg.jend), jg = uniform(guard_from(sg)),
                      keys = uniform(sg.keys);
        const int32_t je[2] = {uniform(sg.je[0]), uniform(sg.je[1])};
        if (jend <= j0) continue;
        tc_wait(bar.q_full, segs & 1, abort, a.err);
        ++segs;
        auto issue_s = [&](int i, uint32_t slot) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((uint32_t)(k >> 2) * L::kPanel + (uint32_t)(k & 3) * 32) >> 4;
                tc_mma_bf16_ss_if(one, tmem + L::kS + i * 128, q_desc + (uint32_t)(i * (L::kTile >> 4) + off),
                                  k_desc + (slot * (L::kTile >> 4) + off), IDESC_S, k > 0 ? 1u : 0u);
            }
            tc_commit_if(one, bar.s_full + 8 * i);
        };
        const uint32_t st = n % L::kStages;
        tc_wait(bar.kv_full + 8 * st, (n / L::kStages) & 1, abort, a.err);
        ++n;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (j0 < je[i]) issue_s(i, st);
        tc_commit_if(one, bar.kv_free + 8 * st);
        if (j0 + 1 == jend) tc_commit_if(one, bar.q_free);
        for (int32_t j = j0; j < jend; ++j) {
            const bool more = j + 1 < jend;
            const uint32_t nv = n, nk = n + 1;  // ring entries of this unit's V and the next one's K
            const uint32_t sv = nv % L::kStages, sk = nk % L::kStages;
            n += more ? 2 : 1;
            tc_wait(bar.kv_full + 8 * sv, (nv / L::kStages) & 1, abort, a.err);
            const bool guarded = j >= jg;
            int ksteps = kTcKeys / 16;
            if (guarded) {
                ksteps = min(ksteps, (keys - j * kTcKeys + 15) / 16);
                if (one) mbar_arrive(bar.v_go);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (j < je[i]) {
                    if (j == j0) {  // O is about to be overwritten: its earlier rows have been read
                        if (no[i] > 0) tc_wait(bar.o_free + 8 * i, (no[i] - 1) & 1, abort, a.err);
                        ++no[i];
                    }
                    tc_wait(bar.p_full + 8 * i, np[i] & 1, abort, a.err);
                    ++np[i];
                }
                if (guarded && i == 0) tc_wait(bar.v_ok, units & 1, abort, a.err);
                if (j < je[i]) {
                    tc_fence_after();
                    auto issue_o = [&](int k) {
                        tc_mma_bf16_ts_if(one, tmem + L::kO + i * D, tmem + L::kS + i * 128 + k * 8,
                                          v_desc + (sv * (L::kTile >> 4) + (uint32_t)k * 128u), IDESC_O,
                                          j > j0 || k > 0 ? 1u : 0u);
                    };
                    if (ksteps == kTcKeys / 16) {
#pragma unroll
                        for (int k = 0; k < kTcKeys / 16; ++k) issue_o(k);
                    } else {
#pragma unroll 1
                        for (int k = 0; k < ksteps; ++k) issue_o(k);
                    }
                    if (j + 1 == je[i]) tc_commit_if(one, bar.o_full + 8 * i);
                }
                if (more && i == 0) tc_wait(bar.kv_full + 8 * sk, (nk / L::kStages) & 1, abort, a.err);
                if (j + 1 < je[i]) {
                    tc_fence_after();
                    issue_s(i, sk);
                }
            }
            if (guarded) ++units;
            tc_commit_if(one, bar.kv_free + 8 * sv);
            if (more) tc_commit_if(one, bar.kv_free + 8 * sk);
            if (j + 2 == jend) tc_commit_if(one, bar.q_free);
        }
    } while (uniform(cur.next(a)));
    // Every MMA ends in an o_full that the softmax warps wait for; nothing of
    // this warp is in flight once they have (see the kernel's end).
}

// ----------------------------------------------------------------- softmax
// Four warps per row tile; a thread owns one query row (tensor-memory lane).
template <int D>
__device__ __forceinline__ void tc_softmax(const PrefillArgs &a, const TcBars &bar, uint32_t tmem,
                                           const OddColumns &odd, int32_t c,
                                           int i, int warp, int lane) {
    using L = TcPrefill<D>;
    const int r = warp * 32 + lane;  // row of the row tile
    const uint32_t t_lane = (uint32_t)(warp * 32) << 16;
    const uint32_t tS = tmem + L::kS + i * 128 + t_lane, tO = tmem + L::kO + i * D + t_lane;
    const uint32_t s_full = bar.s_full + 8 * i, p_full = bar.p_full + 8 * i;
    const int tok_r = r / a.G, g = r - tok_r * a.G;
    const float sl = a.scale_log2;
    uint32_t ns = 0, no = 0, segs = 0;
    bool abort = false;
    PrefillWalk<false> cur;
    if (!cur.init(a, c)) return;
    do {
        const TcSegment sg(a, cur);
        const int32_t tok = i * a.tq1 + tok_r;
        const bool valid = tok_r < a.tq1 && tok < sg.t.ntok;
        const bool warp_rows = __any_sync(0xffffffffu, valid);
        const int32_t last = sg.t.p0 + tok;
        const int32_t je = sg.je[i];
        if (sg.jend > cur.j0) ++segs;
        float m = -INFINITY, l = 0.f;
        for (int32_t j = cur.j0; j < je; ++j) {
            tc_wait(s_full, ns & 1, abort, a.err, a.wait_ns);
            ++ns;
            tc_fence_after();
            if (warp_rows) {
                float x[128];
                tmem_ld_cols(tS, x);
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
                for (int h = 0; h < 4; ++h) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float y0, y1;
                        f32x2_get(fma_f32x2(f32x2(x[32 * h + 2 * k], x[32 * h + 2 * k + 1]), sl2, mm2), y0, y1);
                        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                        sum[k & 1] = add_f32x2(sum[k & 1], f32x2(p0, p1));
                        w[k] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16_async(tS + 16 * h, w);
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
        const bool whole = cur.whole(), out32 = ((uintptr_t)a.out & 31) == 0;
        const int64_t row = cur.slot(c) * (2 * kTcRows) + i * kTcRows + r;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool odd_tile = any && odd.segment[i] == (int32_t)segs;
        __nv_bfloat16 *op =
            (__nv_bfloat16 *)a.out + ((int64_t)(sg.t.row0 + tok) * a.H + (int64_t)cur.kvh * a.G + g) * D;
        if (warp_rows) {
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 64) {
                float o[64];
                if (any) {
                    tmem_ld_cols(tO + (uint32_t)d0, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 64; ++k) o[k] = 0.f;
                }
                if (odd_tile) {
#pragma unroll
                    for (int k = 0; k < 64; ++k) {
                        const int32_t *first = odd.first + d0 + k;
                        if (last >= first[0]) o[k] += INFINITY;
                        if (last >= first[D]) o[k] -= INFINITY;
                        if (last >= first[2 * D]) o[k] += __uint_as_float(0x7fffffffu);
                    }
                }
                if (valid) {
                    // A thread writes a row, so a store's lanes are rows
                    // apart: whole sectors where out's alignment allows.
                    if (whole) {
#pragma unroll
                        for (int k = 0; k < 64; k += 16) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(o[k + 2 * e] * inv, o[k + 2 * e + 1] * inv);
                            if (out32) {
                                store32(op + d0 + k, w);
                            } else {
                                *reinterpret_cast<uint4 *>(op + d0 + k) = make_uint4(w[0], w[1], w[2], w[3]);
                                *reinterpret_cast<uint4 *>(op + d0 + k + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 64; k += 8) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[k + e]);
                            store32(a.acc + row * D + d0 + k, w);
                        }
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
                      const __grid_constant__ CUtensorMap tmv, const __grid_constant__ PrefillArgs a,
                      const int32_t gran) {
    using L = TcPrefill<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const TcBars bar(smem_u32(smem + L::kBars), L::kStages);
    uint32_t *tmem_slot = (uint32_t *)(smem + L::kBars + 248);
    const OddColumns odd{(int32_t *)(smem + L::kBars + 256), (int32_t *)(smem + L::kBars + 240)};
    static_assert(96 + 16 * L::kStages <= 240, "the barriers fit");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(bar.q_full, 1);
        mbar_init(bar.q_free, 1);
        mbar_init(bar.v_go, 1);
        mbar_init(bar.v_ok, 1);
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
        odd.segment[0] = odd.segment[1] = 0;
        fence_mbarrier_init();
    }
    for (int e = tid; e < 3 * D; e += kTcThreads) odd.first[e] = OddColumns::kNone;
    if (warp == 8) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t c = blockIdx.x;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcSoftmaxRegs));
        tc_softmax<D>(a, bar, tmem, odd, c, warp >> 2, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcOtherRegs));
        if (warp == 8)
            tc_issuer<D>(a, smem, bar, tmem, c, lane);
        else if (warp == 9)
            tc_producer<D, false>(a, smem, bar, &tmq, &tmk, gran, c, lane);
        else if (warp == 10)
            tc_producer<D, true>(a, smem, bar, &tmq, &tmv, gran, c, lane);
        else
            tc_guard<D>(a, smem, bar, odd, c, lane);
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
