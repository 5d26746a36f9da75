// Chunk attention on the fifth-generation tensor cores (pa_prefill and pa_cross
// for bf16, pa_prefill_fp8 for an 8-bit cache with a scale per block and KV head;
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
//
// Encoder states (pa_cross): 64 to 448 tokens of 32 sequences over 1000 to 4096
// states (32 / 8 heads, head_dim 128, 258 GFLOP) 226 to 251 us (between boxes, and with the
// power cap); 1 to 8 tokens of 128 sequences over 100 to 1500 (16 heads, head_dim 64, 433
// MB) 114 to 115 us, held by a tile's end every seventh unit or so (over long contexts
// 6.3 TB/s).
#pragma once

#include <cuda.h>  // CUtensorMap

#include "decode_merge.cuh"
#include "fp8_codec.cuh"
#include "prefill_plan.cuh"
#include "tc_ptx.cuh"

namespace pa {

constexpr int kTcRows = 128, kTcKeys = 128, kTcThreads = 384, kTcExtra = 3;
constexpr unsigned long long kTcUnitNs = 4096;
// Registers: 384 threads x 168 at launch; the two softmax warpgroups take 208
// each (a row's 128 scores stay in registers), the third one keeps 88:
// 256 x 208 + 128 x 88 = 384 x 168.
constexpr int kTcSoftmaxRegs = 208, kTcOtherRegs = 88;

// kPair: the form that shares tiles of one row tile (TcSegment), for pa_cross and short
// 8-bit chunks.  pa_prefill, which does not, has a form without that code: with it as a
// run-time choice the same calls took 69.7, 58.5 and 87.5 us (QSlots).
//
// kConv: the warps that turn an 8-bit cache's codes, which arrive in a ring of their
// own (raw), into the bf16 units of the ring that the MMAs read; 0 for a bf16 cache.
// Both forms over an 8-bit cache are right for every call; which one is faster:
//   4  512 threads x 128 registers at launch, 256 x 192 + 128 x 64 + 128 x 64 of them.
//      A row's scores stay in registers.  A unit takes the converters about 1.8 us,
//      two row tiles' softmax and products longer.
//   8  640 x 96, 256 x 112 + 128 x 88 + 256 x 80 and some left.  A unit takes the
//      converters half of that; the softmax, short of registers, reads its scores twice,
//      and shares tiles of one row tile (TcSegment), which leaves it time for that.
// Eight warps where the call's chunks have no more tokens than a row tile on average
// (prefill_layout).  Sequences of 4096 tokens, chunks of 1/8, 1, 1.5 and 4 row tiles, eight
// and four warps in us:
//   64 x, 32 / 8 heads of 128     162 186   169 194   251 230   484 448
//   64 x, 32 / 8 heads of 64      134 158   138 164   221 191   421 361
//   64 x, 16 / 16 heads of 128    309 357   321 374   488 460   926 892
//   64 x, 8 / 1 heads of 128       35  39    38  42    52  49    88  80
//   16 x, 32 / 8 heads of 128      54  61    60  67    85  79   144 133
// 256 sequences of 600, 32 / 8 heads of 128: 163 224, 167 230, 228 261, 433 506: over short
// contexts eight would stay the faster there (heads of 64: 202 206 and 344 312).
template <int D, int kConv, bool kPair>
struct TcPrefill {
    static constexpr bool kFp8 = kConv > 0, kMayPair = kPair;
    static constexpr bool kOneSlot = !kFp8 && !kPair;  // pa_prefill (QSlots)
    static constexpr int kSoftmaxRegs = kConv == 8 ? 112 : kConv == 4 ? 192 : kTcSoftmaxRegs;
    static constexpr int kOtherRegs = kConv == 4 ? 64 : kTcOtherRegs, kConvertRegs = kConv == 8 ? 80 : 64;
    static constexpr int kPanels = D / 64;
    static constexpr uint32_t kPanel = 128 * 128;            // 128 rows of 64 bf16
    static constexpr uint32_t kTile = kPanels * kPanel;      // Q row tile, K or V unit
    static constexpr int kStages = kFp8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);  // ring of K and V units
    static constexpr int kRaw = kFp8 ? (D == 128 ? 4 : 8) : 0;  // units of codes on their way (64 KiB)
    static constexpr uint32_t kRawTile = 128 * D;
    static constexpr int kThreads = kTcThreads + 32 * kConv;
    static constexpr uint32_t kRing = 2 * kTile;             // after the two Q row tiles
    static constexpr uint32_t kRawRing = kRing + kStages * kTile;
    static constexpr uint32_t kBars = kRawRing + kRaw * kRawTile;
    static constexpr uint32_t kBarBytes = (120 + 16 * kStages + 12 + 31) & ~31;  // barriers, OddColumns::segment, the tensor memory's address
    static constexpr uint32_t kRawBars = kBars + kBarBytes + 3 * D * 4;  // barriers; columns with odd values
    static constexpr uint32_t kMl = kRawBars + 16 * kRaw;  // (m, l) of the second warpgroup's rows
    static constexpr uint32_t kMeta = kMl + 1024, kMetaBytes = 40;  // per raw unit: scales of its (up to 16) boxes as bf16, then the number of boxes
    static constexpr uint32_t kBytes = kMeta + kMetaBytes * kRaw;
    static_assert(kBytes <= 227 * 1024, "a CTA's shared memory");
    static constexpr size_t kSmem = kBytes;
    static constexpr uint32_t kS = 0, kO = 256;              // tensor-memory columns: S0, S1, O0, O1
};

// Barriers of a CTA, in shared memory.
struct TcBars {
    uint32_t q_full, q_free, v_go, v_ok, kv_full, kv_free, s_full, p_full, o_full, o_free;  // addresses; arrays 8 bytes apart
    uint32_t x_full, raw_full, raw_free;
    __device__ __forceinline__ TcBars(uint32_t base, int stages, uint32_t raw, int raw_stages) {
        q_full = base;
        q_free = base + 16;
        s_full = base + 32;
        p_full = base + 48;
        o_full = base + 64;
        o_free = base + 80;
        v_go = base + 96;
        v_ok = base + 104;
        x_full = base + 112;
        kv_full = base + 120;
        kv_free = kv_full + 8 * (uint32_t)stages;
        raw_full = raw;
        raw_free = raw + 8 * (uint32_t)raw_stages;
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

// Units of a segment that each row tile takes: [j0, je[i]).  A tile of one row
// tile would leave the second softmax warpgroup idle and wait, unit after unit,
// for its own softmax between two products: with kMayPair the two warpgroups hold
// the same rows and take the units in turn, and the one that had the first unit
// joins the two results at the segment's end.  That one changes from such a
// segment to the next (`first`, counted alike by every role).
template <bool kMayPair>
struct TcSegment {
    PrefillTile t;
    int32_t keys;   // keys the tile sees
    int32_t je[2], jend;
    bool pair;
    // End of row tile i's units.  (An index known only at run time would put the
    // array, and with it every use of it, into memory.)
    __device__ __forceinline__ int32_t end(int i) const { return i ? je[1] : je[0]; }
    // Whether warpgroup i has units of the segment.
    __device__ __forceinline__ bool has(int i, int32_t j0, int first) const {
        return pair ? j0 + (i ^ first) < jend : j0 < end(i);
    }
    template <class Walk>
    __device__ __forceinline__ TcSegment(const PrefillArgs &a, const Walk &cur) {
        t = cur.t;
        keys = prefill_keys(t, t.ntok, a.step);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int32_t n = min(t.ntok, (i + 1) * a.tq1);  // tokens up to this row tile's end
            const int32_t ki = t.ntok > i * a.tq1 ? max(prefill_keys(t, n, a.step), 0) : 0;
            je[i] = min(cur.j1, (int32_t)(((uint32_t)ki + kTcKeys - 1) / kTcKeys));  // the sum may pass 2^31
        }
        jend = max(je[0], je[1]);
        pair = kMayPair && t.ntok <= a.tq1;
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ void sts_u16(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void sts_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ------------------------------------------------------------------ Q slots
// Q's two row tiles in shared memory, each with barriers of its own.  A tile of
// two row tiles takes both; one of a single row tile takes them in turn, so that
// its rows, and the K behind them, are fetched while the tile before is at work
// (long 8-bit chunks 191 -> 184 us).  pa_prefill's form takes both as one slot: a second
// pair of barriers for each of its tiles cost it 4 to 9% on short contexts (16 x 400
// tokens, 32 / 8 heads: 62.2 and 65.7 us at head_dim 128, 51.0 and 53.0 at 64; 64 x 40
// over 1000 79.6 and 86.3).  The K producer and the issuer count alike.
struct QSlots {
    uint32_t n0 = 0, n1 = 0;  // tiles that each slot has held
    int next = 0;             // the slot of the next tile of a single row tile
    __device__ __forceinline__ uint32_t &n(int s) { return s ? n1 : n0; }
};
// K producer: waits for the slots of a tile's rows and fetches them.
template <class L>
__device__ __forceinline__ void load_q(const PrefillArgs &a, const PrefillTile &t, int32_t kvh, uint32_t q_dst,
                                       const TcBars &bar, const CUtensorMap *tmq, QSlots &q, bool &abort, int lane) {
    const bool two = t.ntok > a.tq1;
    auto wait = [&](int s) {
        if (q.n(s) > 0) tc_wait(bar.q_free + 8 * s, (q.n(s) - 1) & 1, abort, a.err);
        ++q.n(s);
        return !__any_sync(0xffffffffu, abort);
    };
    auto load = [&](int slot, uint32_t full, int32_t row) {
        for (int32_t p = 0; p < L::kPanels; ++p)
            tma_load_4d(q_dst + slot * L::kTile + p * L::kPanel, tmq, full, 0, p, kvh * a.G, row);
    };
    const uint32_t bytes = (uint32_t)(L::kPanels * a.tq1 * a.G) * 128u;  // of a row tile
    if constexpr (L::kOneSlot) {
        if (!wait(0)) return;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar.q_full, two ? 2 * bytes : bytes);
            for (int32_t i = 0; i < (two ? 2 : 1); ++i) load(i, bar.q_full, t.row0 + i * a.tq1);
        }
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (!two && s != q.next) continue;
            if (!wait(s)) return;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar.q_full + 8 * s, bytes);
                load(s, bar.q_full + 8 * s, t.row0 + (two ? s * a.tq1 : 0));
            }
        }
        if (!two) q.next ^= 1;
    }
}
// The last fetches and the issuer's last arrivals on the free barriers.
__device__ __forceinline__ void drain_q(const TcBars &bar, QSlots &q, bool &late, unsigned int *err) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (q.n(s) == 0) continue;
        tc_wait(bar.q_full + 8 * s, (q.n(s) - 1) & 1, late, err);
        tc_wait(bar.q_free + 8 * s, (q.n(s) - 1) & 1, late, err);
    }
}

// ----------------------------------------------------------- TMA producers
// One warp for K (and the Q rows), one for V.  Entry n of the ring is K of a
// unit for even n, V for odd n.  A unit is 128 / gran boxes per panel, gran =
// gcd(block size, 128) keys, one box per lane; the block-table entry of a
// lane's next box is read a unit ahead and looked at when its unit comes, so
// no load is waited for.  Q: one box of tq1 tokens x G heads per row tile and
// 64-element panel.
template <int D, bool kPair, bool kIsV>
__device__ __forceinline__ void tc_producer(const PrefillArgs &a, uint8_t *smem, const TcBars &bar,
                                            const CUtensorMap *tmq, const CUtensorMap *tm, int32_t gran,
                                            int32_t c, int lane) {
    using L = TcPrefill<D, 0, kPair>;
    if (lane == 0) {
        if (!kIsV) prefetch_tmap(tmq);
        prefetch_tmap(tm);
    }
    const uint32_t q_dst = smem_u32(smem), ring = q_dst + L::kRing;
    const int32_t nbm = kTcKeys / gran;  // boxes of a unit per panel (at most 16)
    const int32_t bi = lane % nbm, panel = lane / nbm;
    const bool has_box = panel < L::kPanels;
    const uint32_t box_off = (uint32_t)panel * L::kPanel + (uint32_t)(bi * gran) * 128u;
    uint32_t n = kIsV ? 1 : 0;  // next ring entry
    QSlots q;
    bool abort = false;
    PrefillCursor cur;
    if (!cur.init(a, c)) return;
    do {
        const TcSegment<L::kMayPair> sg(a, cur);
        if (sg.jend <= cur.j0) continue;
        const int32_t *row = a.tables + (int64_t)sg.t.seq * a.max_blocks;
        auto has_key = [&](int32_t j) { return has_box && (int64_t)j * kTcKeys + bi * gran < sg.keys; };
        auto entry = [&](int32_t j) { return has_key(j) ? row[(j * kTcKeys + bi * gran) / a.B] : 0; };
        int32_t phys = entry(cur.j0);
        if (!kIsV) {
            load_q<L>(a, sg.t, cur.kvh, q_dst, bar, tmq, q, abort, lane);
            if (__any_sync(0xffffffffu, abort)) break;
        }
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
    if (!kIsV) drain_q(bar, q, late, a.err);
}

// ------------------------------------------------- 8-bit cache: producers
// As above, but an entry n is 128 rows of D codes in the raw ring, a box one
// block's rows (gran of them), with the box's scale byte brought by its lane: the
// byte is asked for a unit ahead, the table entry two.  The K warp ends the
// ring with an entry of kRawEnd boxes, at which the converters stop.
constexpr int32_t kRawEnd = -1;

// Ring entry of unit u's K and V, of n units that a segment begins with at entry 0.
// Over the 8-bit cache, whose rings are short, a pair's entries come in the order
// of their use, K0 K1 V0 K2 V1 .. (the next but one S follows an O): with K and V
// in turn, K would wait for the slot of a V that has just been used.  Everything
// else takes K and V in turn.
template <bool kFp8>
__device__ __forceinline__ uint32_t k_entry(bool pair, int32_t u) {
    return kFp8 && pair && u > 0 ? 2u * (uint32_t)u - 1u : 2u * (uint32_t)u;
}
template <bool kFp8>
__device__ __forceinline__ uint32_t v_entry(bool pair, int32_t u, int32_t n) {
    return kFp8 && pair && u + 1 < n ? 2u * (uint32_t)u + 2u : 2u * (uint32_t)u + 1u;
}

template <int D, int kConv, bool kPair, bool kIsV>
__device__ __forceinline__ void tc_producer8(const PrefillArgs &a, uint8_t *smem, const TcBars &bar,
                                             const CUtensorMap *tmq, const CUtensorMap *tm, int32_t gran,
                                             int32_t c, int lane) {
    using L = TcPrefill<D, kConv, kPair>;
    if (lane == 0) {
        if (!kIsV) prefetch_tmap(tmq);
        prefetch_tmap(tm);
    }
    const uint32_t q_dst = smem_u32(smem), raw = q_dst + L::kRawRing, meta = q_dst + L::kMeta;
    const int32_t nbm = kTcKeys / gran;  // boxes of a unit (at most 16), one per lane
    const uint8_t *scales = kIsV ? a.v_scale : a.k_scale;
    const uint64_t policy = l2_policy_evict_first();
    uint32_t base = 0;  // entries of the segments before
    QSlots q;
    bool abort = false;
    PrefillWalk<false> cur;
    if (cur.init(a, c)) {
        do {
            const TcSegment<L::kMayPair> sg(a, cur);
            if (sg.jend <= cur.j0) continue;
            const int32_t *row = a.tables + (int64_t)sg.t.seq * a.max_blocks;
            auto has_key = [&](int32_t j) { return lane < nbm && (int64_t)j * kTcKeys + lane * gran < sg.keys; };
            auto entry = [&](int32_t j) { return j < sg.jend && has_key(j) ? row[(j * kTcKeys + lane * gran) / a.B] : 0; };
            auto scale_at = [&](int32_t p) -> uint32_t {  // a bad entry: the smallest scale, of codes that are zeros
                return lane < nbm && p >= 0 && p < a.NB ? scales[(int64_t)p * a.Hk + cur.kvh] : 0u;
            };
            int32_t phys = entry(cur.j0), phys_1 = entry(cur.j0 + 1);
            if (!kIsV) {
                load_q<L>(a, sg.t, cur.kvh, q_dst, bar, tmq, q, abort, lane);
                if (__any_sync(0xffffffffu, abort)) break;
            }
            uint32_t sc = scale_at(phys);
            const int32_t nu = sg.jend - cur.j0;
            for (int32_t j = cur.j0; j < sg.jend; ++j) {
                const uint32_t n = base + (kIsV ? v_entry<true>(sg.pair, j - cur.j0, nu) : k_entry<true>(sg.pair, j - cur.j0));
                const bool box = has_key(j);
                int32_t at = a.NB * a.B;  // a bad entry reads zeros: the box lies past the pool
                if (phys >= 0 && phys < a.NB)
                    at = phys * a.B + (j * kTcKeys + lane * gran) % a.B;
                else if (box)
                    atomicOr(a.err, kErrBounds);
                const uint32_t sc_now = sc;
                phys = phys_1;
                sc = scale_at(phys);
                phys_1 = entry(j + 2);
                const uint32_t boxes = (uint32_t)__popc(__ballot_sync(0xffffffffu, box));
                const uint32_t st = n % L::kRaw;
                if (n >= L::kRaw) tc_wait(bar.raw_free + 8 * st, (n / L::kRaw + 1) & 1, abort, a.err);
                if (__any_sync(0xffffffffu, abort)) break;
                if (box) sts_u16(meta + st * L::kMetaBytes + (uint32_t)lane * 2, __float_as_uint(scale_of(sc_now)) >> 16);
                if (lane == 0) sts_u32(meta + st * L::kMetaBytes + 32, boxes);
                __syncwarp();  // in place before lane 0 publishes the entry
                if (lane == 0) mbar_arrive_expect_tx(bar.raw_full + 8 * st, boxes * (uint32_t)gran * D);
                __syncwarp();
                if (box)
                    tma_load_3d_hint(raw + st * L::kRawTile + (uint32_t)(lane * gran) * D, tm, bar.raw_full + 8 * st, 0, at,
                                     cur.kvh, policy);
            }
            base += 2 * (uint32_t)nu;
            if (__any_sync(0xffffffffu, abort)) break;
        } while (cur.next(a));
    }
    // Every copy lands before the converters, which wait for each entry, come to the
    // end entry.  After a wait that ran out, look at the last ones here.
    bool late = false;
    if (abort)
        for (uint32_t k = base > (uint32_t)L::kRaw ? base - L::kRaw : 0; k < base; ++k)
            tc_wait(bar.raw_full + 8 * (k % L::kRaw), (k / L::kRaw) & 1, late, a.err);
    if (!kIsV) {
        const uint32_t st = base % L::kRaw;
        if (base >= L::kRaw) tc_wait(bar.raw_free + 8 * st, (base / L::kRaw + 1) & 1, abort, a.err);
        if (lane == 0 && !abort) {
            sts_u32(meta + st * L::kMetaBytes + 32, (uint32_t)kRawEnd);
            mbar_arrive(bar.raw_full + 8 * st);
        }
        // the issuer's last arrivals on the free barriers land before the CTA may exit
        for (uint32_t k = base > (uint32_t)L::kStages ? base - L::kStages : 0; k < base; ++k)
            tc_wait(bar.kv_free + 8 * (k % L::kStages), (k / L::kStages) & 1, late, a.err);
    }
    if (!kIsV) drain_q(bar, q, late, a.err);
}

// ------------------------------------------------------- 8-bit: converters
// kConv warps turn entry n of the raw ring into entry n of the bf16 ring: code *
// 2^(byte - 127), in fp32 and then bf16 (one rounding, of values that bf16 holds
// exactly unless they leave its range).  Per two codes: a conversion to fp16, two
// to fp32, a packed product, a packed conversion.  (Shifting codes into place as bf16 and one packed bf16 product
// took as many instructions with the look for NaN codes, and longer.)
// A thread takes 16 codes at a time (a 16-byte load) and stores them as two
// 16-byte chunks of a swizzled 128-byte line.  Eight lanes' loads and stores fall
// into distinct banks: at head_dim 128 they hold four pieces each of rows r and r ^ 5,
// whose swizzles differ in both the bit that parts the halves of a line of codes
// and the one that parts even from odd chunks; at head_dim 64 of rows r and r + 1.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint64_t s2, uint32_t &lo, uint32_t &hi) {
    uint32_t a, b;
    codes_f16(w, a, b);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a)), y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    float u, v;
    f32x2_get(mul_f32x2(f32x2(x.x, x.y), s2), u, v);
    lo = pack_bf16x2(u, v);
    f32x2_get(mul_f32x2(f32x2(y.x, y.y), s2), u, v);
    hi = pack_bf16x2(u, v);
}

template <int D, int kConv, bool kPair>
__device__ __forceinline__ void tc_converter(const PrefillArgs &a, uint8_t *smem, const TcBars &bar, int32_t gran, int tid) {
    using L = TcPrefill<D, kConv, kPair>;
    constexpr int kRowsPass = (D == 128 ? 4 : 8) * kConv;  // rows of the warps at once
    constexpr int kPasses = 128 / kRowsPass, kBatch = 2;  // loads of a thread in flight
    const uint32_t raw = smem_u32(smem) + L::kRawRing, ring = smem_u32(smem) + L::kRing;
    const uint32_t meta = smem_u32(smem) + L::kMeta;
    const int lane = tid & 31;
    const int shift = __ffs(gran) - 1;  // gran = gcd(block size, 128)
    // D 128: half of the warps take the first panel, the others the second
    const int r0 = D == 128 ? ((tid >> 2) & (kRowsPass - 8)) | (((tid >> 3) & 3) ^ (tid & 4 ? 5 : 0)) : tid >> 2;
    const uint32_t panel = D == 128 ? (uint32_t)tid / (16u * kConv) : 0u, ch = (uint32_t)tid & 3u;
    const uint32_t src = D == 128 ? (uint32_t)r0 * 128u + (((panel * 4u + ch) ^ (uint32_t)(r0 & 7)) << 4) : (uint32_t)tid * 16u;
    // rows of a thread are a multiple of 8 apart: their swizzle is the same
    const uint32_t dst = panel * L::kPanel + (uint32_t)r0 * 128u + (((ch * 2u) ^ (uint32_t)(r0 & 7)) << 4);
    bool abort = false;
    for (uint32_t n = 0;; ++n) {
        const uint32_t rs = n % L::kRaw, st = n % L::kStages;
        tc_wait(bar.raw_full + 8 * rs, (n / L::kRaw) & 1, abort, a.err, a.wait_ns);
        const int32_t boxes = (int32_t)lds_u32(meta + rs * L::kMetaBytes + 32);
        if (__any_sync(0xffffffffu, abort || boxes == kRawEnd)) break;
        if (n >= L::kStages) tc_wait(bar.kv_free + 8 * st, (n / L::kStages + 1) & 1, abort, a.err, a.wait_ns);
        if (__any_sync(0xffffffffu, abort)) break;
        const int32_t rows = boxes * gran;
        const uint32_t from = raw + rs * L::kRawTile + src, to = ring + st * L::kTile + dst, scales = meta + rs * L::kMetaBytes;
        auto scale = [&](int p) { return lds_bf16(scales + (uint32_t)(((p * kRowsPass + r0) >> shift) * 2)); };
        uint4 w[kBatch];
        float s[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) w[b] = lds128(from + (uint32_t)b * (kRowsPass * D)), s[b] = scale(b);
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {  // rows past the boxes: whatever the ring holds
            if (p % kBatch == 0 && p * kRowsPass >= rows) break;
            const uint4 v = w[p % kBatch];
            const uint64_t s2 = f32x2(s[p % kBatch], s[p % kBatch]);
            if (p + kBatch < kPasses) {
                w[p % kBatch] = lds128(from + (uint32_t)(p + kBatch) * (kRowsPass * D));
                s[p % kBatch] = scale(p + kBatch);
            }
            uint4 x, y;
            codes_bf16(v.x, s2, x.x, x.y);
            codes_bf16(v.y, s2, x.z, x.w);
            codes_bf16(v.z, s2, y.x, y.y);
            codes_bf16(v.w, s2, y.z, y.w);
            const uint32_t at = to + (uint32_t)p * (kRowsPass * 128);
            sts128(at, x);
            sts128(at ^ 16u, y);
        }
        fence_proxy_async_smem();  // the MMAs read the unit through the async proxy
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar.kv_full + 8 * st);
            mbar_arrive(bar.raw_free + 8 * rs);
        }
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
template <class Segment>
__device__ __forceinline__ int32_t guard_from(const Segment &sg) { return max(sg.t.p0 + 1, 0) / kTcKeys; }

template <int D>
__device__ __forceinline__ uint32_t v_chunk(uint32_t vbase, int e) {  // address of 16-byte chunk e % (D / 8) of row e / (D / 8)
    constexpr int kChunks = D / 8;
    const int r = e / kChunks, ch = e % kChunks;
    return vbase + (uint32_t)(ch >> 3) * TcPrefill<D, 0, false>::kPanel + (uint32_t)r * 128u +
           (uint32_t)(((ch & 7) ^ (r & 7)) << 4);
}
// Sign bits of the halves whose exponent is all ones (bf16 infinities and NaN).
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

template <int D, int kConv, bool kPair>
__device__ __forceinline__ void tc_guard(const PrefillArgs &a, uint8_t *smem, const TcBars &bar, const OddColumns &odd,
                                         int32_t c, int lane) {
    using L = TcPrefill<D, kConv, kPair>;
    constexpr int kChunks = D / 8;
    const uint32_t ring = smem_u32(smem) + L::kRing;
    uint32_t n = 0, segs = 0, units = 0;  // ring entries of the segments before, segments, guarded units
    uint32_t no[2] = {0, 0};              // earlier segments with units per row tile
    uint32_t held = 0;                    // the segment that the columns belong to
    int first = 0;                        // (TcSegment)
    bool abort = false;
    PrefillCursor cur;
    const bool work = cur.init(a, c);
    if (lane == 0) note_cut(a, c, work, cur);
    if (!work) return;
    do {
        const TcSegment<L::kMayPair> sg(a, cur);
        if (sg.jend <= cur.j0) continue;
        ++segs;
        for (int32_t j = max(cur.j0, guard_from(sg)); j < sg.jend; ++j, ++units) {
            // The issuer has seen V arrive.  This wait and the softmax's for S
            // may last while the other roles work through most of the CTA's
            // range, so their limit grows with the range.
            tc_wait(bar.v_go, units & 1, abort, a.err, a.wait_ns);
            const uint32_t vbase =
                ring + (n + v_entry<L::kFp8>(sg.pair, j - cur.j0, sg.jend - cur.j0)) % L::kStages * L::kTile;
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
                    if (no[i] > 0 && (sg.pair || j == cur.j0 || sg.je[i] <= cur.j0))
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
        for (int i = 0; i < 2; ++i) no[i] += sg.has(i, cur.j0, first) ? 1 : 0;
        if (sg.pair) first ^= 1;
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
template <int D, int kConv, bool kPair>
__device__ __forceinline__ void tc_issuer(const PrefillArgs &a, uint8_t *smem, const TcBars &bar, uint32_t tmem,
                                          int32_t c, int lane) {
    using L = TcPrefill<D, kConv, kPair>;
    constexpr uint32_t IDESC_S = tc_idesc_bf16(128, kTcKeys, false, false);
    constexpr uint32_t IDESC_O = tc_idesc_bf16(128, D, false, true);
    const uint32_t ring = smem_u32(smem) + L::kRing;
    // Descriptors of the first Q row tile and ring entry; the others' start
    // addresses (in 16-byte units, the low bits of a descriptor) are added.
    const uint64_t q_desc = smem_desc_sw128(smem_u32(smem), 16, 1024), k_desc = smem_desc_sw128(ring, 16, 1024),
                   v_desc = smem_desc_sw128(ring, L::kPanel, 1024);
    const uint32_t one = elect_one();
    uint32_t n = 0, units = 0;  // ring entries consumed, guarded units
    QSlots qs;
    uint32_t np[2] = {0, 0};              // P tiles taken per row tile
    uint32_t no[2] = {0, 0};              // segments with units per row tile
    int first = 0;                        // (TcSegment)
    bool abort = false;
    PrefillCursor cur;
    if (!cur.init(a, c)) return;
    do {
        const TcSegment<L::kMayPair> sg(a, cur);
        const int32_t j0 = uniform(cur.j0), jend = uniform(sg.jend), jg = uniform(guard_from(sg)),
                      keys = uniform(sg.keys);
        const int32_t je[2] = {uniform(sg.je[0]), uniform(sg.je[1])};
        const bool pair = L::kMayPair && uniform(sg.pair) != 0;
        if (jend <= j0) continue;
        const bool two = L::kOneSlot || uniform(sg.t.ntok > a.tq1) != 0;
        const int q0 = L::kOneSlot ? 0 : uniform(two ? 0 : qs.next);  // Q's slot of the first row tile
#pragma unroll
        for (int s = 0; s < (L::kOneSlot ? 1 : 2); ++s)
            if (two || s == q0) {
                tc_wait(bar.q_full + 8 * s, qs.n(s) & 1, abort, a.err);
                ++qs.n(s);
            }
        if (!two) qs.next ^= 1;
        auto free_q = [&]() {
#pragma unroll
            for (int s = 0; s < (L::kOneSlot ? 1 : 2); ++s)
                if (two || s == q0) tc_commit_if(one, bar.q_free + 8 * s);
        };
        auto issue_s = [&](int i, uint32_t slot, int q) {  // slot q of Q
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((uint32_t)(k >> 2) * L::kPanel + (uint32_t)(k & 3) * 32) >> 4;
                tc_mma_bf16_ss_if(one, tmem + L::kS + i * 128, q_desc + (uint32_t)(q * (L::kTile >> 4) + off),
                                  k_desc + (slot * (L::kTile >> 4) + off), IDESC_S, k > 0 ? 1u : 0u);
            }
            tc_commit_if(one, bar.s_full + 8 * i);
        };
        if (pair) {  // the warpgroups take the units in turn, both with Q's first row tile
            const uint32_t base = n;
            n += 2 * (uint32_t)(jend - j0);
            auto s_of = [&](int i, int32_t j) {
                const uint32_t ek = base + k_entry<L::kFp8>(true, j - j0), sk = ek % L::kStages;
                tc_wait(bar.kv_full + 8 * sk, (ek / L::kStages) & 1, abort, a.err);
                tc_fence_after();
                issue_s(i, sk, q0);
                tc_commit_if(one, bar.kv_free + 8 * sk);
                if (j + 1 == jend) free_q();
            };
            int i = first;  // warpgroup of unit j
            s_of(i, j0);
            if (j0 + 1 < jend) s_of(i ^ 1, j0 + 1);
            first ^= 1;
#pragma unroll 1
            for (int32_t j = j0; j < jend; ++j, i ^= 1) {
                const uint32_t ev = base + v_entry<L::kFp8>(true, j - j0, jend - j0), sv = ev % L::kStages;
                tc_wait(bar.kv_full + 8 * sv, (ev / L::kStages) & 1, abort, a.err);
                const bool guarded = j >= jg;
                int ksteps = kTcKeys / 16;
                if (guarded) {
                    ksteps = min(ksteps, (keys - j * kTcKeys + 15) / 16);
                    if (one) mbar_arrive(bar.v_go);
                }
                const bool begins = j < j0 + 2;
                if (begins) {  // O is about to be overwritten: its earlier rows have been read
                    const uint32_t k = i ? no[1]++ : no[0]++;
                    if (k > 0) tc_wait(bar.o_free + 8 * i, (k - 1) & 1, abort, a.err);
                }
                tc_wait(bar.p_full + 8 * i, (i ? np[1]++ : np[0]++) & 1, abort, a.err);
                if (guarded) {
                    tc_wait(bar.v_ok, units & 1, abort, a.err);
                    ++units;
                }
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < ksteps; ++k)
                    tc_mma_bf16_ts_if(one, tmem + L::kO + i * D, tmem + L::kS + i * 128 + k * 8,
                                      v_desc + (sv * (L::kTile >> 4) + (uint32_t)k * 128u), IDESC_O,
                                      !begins || k > 0 ? 1u : 0u);
                if (j + 2 >= jend) tc_commit_if(one, bar.o_full + 8 * i);
                tc_commit_if(one, bar.kv_free + 8 * sv);
                if (j + 2 < jend) s_of(i, j + 2);
            }
            continue;
        }
        const uint32_t st = n % L::kStages;
        tc_wait(bar.kv_full + 8 * st, (n / L::kStages) & 1, abort, a.err);
        ++n;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (j0 < je[i]) issue_s(i, st, two ? i : q0);
        tc_commit_if(one, bar.kv_free + 8 * st);
        if (j0 + 1 == jend) free_q();
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
                    issue_s(i, sk, two ? i : q0);
                }
            }
            if (guarded) ++units;
            tc_commit_if(one, bar.kv_free + 8 * sv);
            if (more) tc_commit_if(one, bar.kv_free + 8 * sk);
            if (j + 2 == jend) free_q();
        }
    } while (uniform(cur.next(a)));
    // Every MMA ends in an o_full that the softmax warps wait for; nothing of
    // this warp is in flight once they have (see the kernel's end).
}

// A row's O out of tensor memory, with the other warpgroup's where there is one
// (tO_other; w0 and w1 their weights), and with the values that are not finite that
// the row sees (odd): to out, or to the segment's piece
// with (m, l).
template <int D, class Walk, class Segment>
__device__ __forceinline__ void write_rows(const PrefillArgs &a, const Walk &cur, int32_t c, const Segment &sg, int i, int r,
                                           int32_t tok, int g, bool valid, int32_t last, bool any, const int32_t *odd,
                                           uint32_t tO, float w0, uint32_t tO_other, float w1, float m, float l) {
    const bool whole = cur.whole(), out32 = ((uintptr_t)a.out & 31) == 0;
    const int64_t row = cur.slot(c) * (2 * kTcRows) + (sg.pair ? 0 : i) * kTcRows + r;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16 *op = (__nv_bfloat16 *)a.out + ((int64_t)(sg.t.row0 + tok) * a.H + (int64_t)cur.kvh * a.G + g) * D;
    __syncwarp();  // converged, as the tensor memory's loads want it
    // 16 columns at a time in a short loop: this code runs once per segment, and
    // unrolled over a row most of its time was its own fetching
    // (68 sequences of 1 to 130 tokens over 1 to 1664 states: 120 and 115 us).
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += 16) {
        float o[16];
        if (any) {
            tmem_ld16(tO + (uint32_t)d0, o);
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0.f;
        }
        if (tO_other) {
            float y[16];
            tmem_ld16(tO_other + (uint32_t)d0, y);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = fmaf(w1, y[k], w0 * o[k]);
        }
        if (odd) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int32_t *first = odd + d0 + k;
                if (last >= first[0]) o[k] += INFINITY;
                if (last >= first[D]) o[k] -= INFINITY;
                if (last >= first[2 * D]) o[k] += __uint_as_float(0x7fffffffu);
            }
        }
        // A thread writes a row, so a store's lanes are rows apart: whole sectors
        // where out's alignment allows.  Predicated, so that the warp stays
        // converged for the next load.
        if (whole) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
            if (out32) {
                store32_if(valid, op + d0, w);
            } else {
                store16_if(valid, op + d0, make_uint4(w[0], w[1], w[2], w[3]));
                store16_if(valid, op + d0 + 8, make_uint4(w[4], w[5], w[6], w[7]));
            }
        } else {
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[k + e]);
                store32_if(valid, a.acc + row * D + d0 + k, w);
            }
        }
    }
    if (valid && !whole) a.ml[row] = make_float2(m, l);
}

// ----------------------------------------------------------------- softmax
// Four warps per row tile; a thread owns one query row (tensor-memory lane).
template <int D, int kConv, bool kPair>
__device__ __forceinline__ void tc_softmax(const PrefillArgs &a, const TcBars &bar, uint32_t tmem,
                                           const OddColumns &odd, float2 *ml, int32_t c,
                                           int i, int warp, int lane) {
    using L = TcPrefill<D, kConv, kPair>;
    const int r = warp * 32 + lane;  // row of the row tile
    const uint32_t t_lane = (uint32_t)(warp * 32) << 16;
    const uint32_t tS = tmem + L::kS + i * 128 + t_lane, tO = tmem + L::kO + i * D + t_lane, tO_other = tmem + L::kO + (1 - i) * D + t_lane;
    const uint32_t s_full = bar.s_full + 8 * i, p_full = bar.p_full + 8 * i;
    const int tok_r = r / a.G, g = r - tok_r * a.G;
    const float sl = a.scale_log2;
    uint32_t ns = 0, no = 0, segs = 0, nx = 0;
    int first = 0;
    bool abort = false;
    PrefillWalk<false> cur;
    if (!cur.init(a, c)) return;
    do {
        const TcSegment<L::kMayPair> sg(a, cur);
        const int32_t tok = (sg.pair ? 0 : i * a.tq1) + tok_r;
        const bool valid = tok_r < a.tq1 && tok < sg.t.ntok;
        const bool warp_rows = __any_sync(0xffffffffu, valid);
        const int32_t last = sg.t.p0 + a.step * tok;  // last key that this row sees
        // This warpgroup's units: every one of its row tile's, or every other one.
        const int32_t je = sg.pair ? sg.jend : sg.end(i), jf = cur.j0 + (sg.pair ? i ^ first : 0), dj = sg.pair ? 2 : 1;
        const bool second = sg.pair && i != first;
        if (sg.pair && sg.jend > cur.j0) first ^= 1;
        if (sg.jend > cur.j0) ++segs;
        float m = -INFINITY, l = 0.f;
        for (int32_t j = jf; j < je; j += dj) {
            tc_wait(s_full, ns & 1, abort, a.err, a.wait_ns);
            ++ns;
            tc_fence_after();
            if (warp_rows) {
                const int32_t nvis = last - j * kTcKeys + 1;
                const bool masked = __any_sync(0xffffffffu, valid && nvis < kTcKeys);
                // A row's scores in registers, all 128 or (beside eight converter warps,
                // for want of registers) 32 at a time, read twice.
                constexpr int kCols = kConv == 8 ? 32 : 128;
                float x[kCols];
                auto read = [&](int h) {
                    if constexpr (kCols == 32)
                        tmem_ld32(tS + kCols * h, x);
                    else
                        tmem_ld_cols(tS + kCols * h, x);
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < kCols; ++k) x[k] = kCols * h + k < nvis ? x[k] : -INFINITY;
                    }
                };
                float top = -INFINITY;
#pragma unroll 1
                for (int h = 0; h < 128 / kCols; ++h) {
                    read(h);
                    float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int k = 4; k < kCols; k += 8) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            mx[q] = k + q + 4 < kCols ? fmaxf(fmaxf(mx[q], x[k + q]), x[k + q + 4]) : fmaxf(mx[q], x[k + q]);
                    }
                    top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                }
                top *= sl;
                // Lazy running maximum: moved (with l and O rescaled) only when
                // a score passes it by more than kLazyMaxSlack.
                const bool grow = valid && top > m + kLazyMaxSlack;
                if (__any_sync(0xffffffffu, grow)) {
                    const float mn = grow ? top : m;
                    const float al = grow ? ex2_approx(m - mn) : 1.f;
                    m = mn;
                    l *= al;
                    if (j > jf) {
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
                auto weigh = [&](int h, int at) {  // columns 32 h .., in x from `at` on
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float y0, y1;
                        f32x2_get(fma_f32x2(f32x2(x[at + 2 * k], x[at + 2 * k + 1]), sl2, mm2), y0, y1);
                        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                        sum[k & 1] = add_f32x2(sum[k & 1], f32x2(p0, p1));
                        w[k] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16_async(tS + 16 * h, w);  // over columns that have been read
                };
                if constexpr (kCols == 32) {
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        read(h);
                        weigh(h, 0);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h) weigh(h, 32 * h);
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
        const bool any = je > jf;
        if (any) {
            tc_wait(bar.o_full + 8 * i, no & 1, abort, a.err);
            ++no;
            tc_fence_after();
        }
        if (second) {  // the other warpgroup takes over: it reads both O, and frees them
            if (any) {
                ml[r] = make_float2(m, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.x_full);
                ++nx;
            }
            continue;
        }
        const bool join = sg.pair && cur.j0 + 1 < sg.jend;
        float w0 = 1.f, w1 = 0.f;
        if (join) {
            tc_wait(bar.x_full, nx & 1, abort, a.err);
            ++nx;
            tc_fence_after();
            const float2 y = ml[r];
            const float mn = fmaxf(m, y.x), mref = mn == -INFINITY ? 0.f : mn;  // a row without keys: zeros
            w0 = ex2_approx(m - mref), w1 = ex2_approx(y.x - mref);
            l = w0 * l + w1 * y.y;
            m = mn;
        }
        const bool odd_tile = any && odd.segment[sg.pair ? 0 : i] == (int32_t)segs;
        if (warp_rows)
            write_rows<D>(a, cur, c, sg, i, r, tok, g, valid, last, any, odd_tile ? odd.first : nullptr, tO, w0,
                          join ? tO_other : 0u, w1, m, l);
        if (any) {  // O (and the odd columns) have been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.o_free + 8 * i);
            if (lane == 0 && join) mbar_arrive(bar.o_free + 8 * (1 - i));
        }
    } while (cur.next(a));
}

template <int D, int kConv, bool kPair>
__global__ void __launch_bounds__(TcPrefill<D, kConv, kPair>::kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const __grid_constant__ PrefillArgs a,
                      const int32_t gran) {
    using L = TcPrefill<D, kConv, kPair>;
    extern __shared__ __align__(1024) uint8_t smem_tc[];
    uint8_t *smem = smem_tc;
    if ((smem_u32(smem) & 1023) != 0) {  // no room to align it here (the layout fills the CTA's limit)
        if (threadIdx.x == 0) atomicOr(a.err, kErrTimeout);
        return;
    }
    const TcBars bar(smem_u32(smem + L::kBars), L::kStages, smem_u32(smem + L::kRawBars), L::kRaw);
    uint32_t *tmem_slot = (uint32_t *)(smem + L::kBars + 128 + 16 * L::kStages);
    const OddColumns odd{(int32_t *)(smem + L::kBars + L::kBarBytes), (int32_t *)(smem + L::kBars + 120 + 16 * L::kStages)};

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(bar.v_go, 1);
        mbar_init(bar.v_ok, 1);
        mbar_init(bar.x_full, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar.q_full + 8 * i, 1);
            mbar_init(bar.q_free + 8 * i, 1);
            mbar_init(bar.s_full + 8 * i, 1);
            mbar_init(bar.p_full + 8 * i, 4);
            mbar_init(bar.o_full + 8 * i, 1);
            mbar_init(bar.o_free + 8 * i, 4);
        }
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar.kv_full + 8 * s, L::kFp8 ? kConv : 1);
            mbar_init(bar.kv_free + 8 * s, 1);
        }
        for (int s = 0; s < L::kRaw; ++s) {
            mbar_init(bar.raw_full + 8 * s, 1);
            mbar_init(bar.raw_free + 8 * s, kConv);
        }
        odd.segment[0] = odd.segment[1] = 0;
        fence_mbarrier_init();
    }
    for (int e = tid; e < 3 * D; e += L::kThreads) odd.first[e] = OddColumns::kNone;
    if (warp == 8) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t c = blockIdx.x;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoftmaxRegs));
        tc_softmax<D, kConv, kPair>(a, bar, tmem, odd, (float2 *)(smem + L::kMl), c, warp >> 2, warp & 3, lane);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kOtherRegs));
        if (warp == 8) {
            tc_issuer<D, kConv, kPair>(a, smem, bar, tmem, c, lane);
        } else if (warp == 9) {
            if constexpr (L::kFp8)
                tc_producer8<D, kConv, kPair, false>(a, smem, bar, &tmq, &tmk, gran, c, lane);
            else
                tc_producer<D, kPair, false>(a, smem, bar, &tmq, &tmk, gran, c, lane);
        } else if (warp == 10) {
            if constexpr (L::kFp8)
                tc_producer8<D, kConv, kPair, true>(a, smem, bar, &tmq, &tmv, gran, c, lane);
            else
                tc_producer<D, kPair, true>(a, smem, bar, &tmq, &tmv, gran, c, lane);
        } else {
            tc_guard<D, kConv, kPair>(a, smem, bar, odd, c, lane);
        }
    } else if constexpr (L::kFp8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kConvertRegs));
        tc_converter<D, kConv, kPair>(a, smem, bar, gran, tid - 384);
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
