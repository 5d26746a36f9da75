// Work list, pieces and merge of chunk attention (pa_prefill).
//
// The chunk's new tokens are cut into tiles of tq tokens x the G query heads
// of one KV head; a tile attends to keys 0 .. p0 + ntok - 1 of its sequence
// in units of kt keys.  A tile weighs its units plus `extra`, the cost of
// beginning and ending one in units (Q's load, the pipeline's ramp, the
// output), laid before its units; the flattened list of (KV head, tile,
// weight) is cut evenly over C persistent CTAs (split_begin), so that long and
// short chunks, and one long context as well as many short ones, load every
// CTA alike.  A CTA's range is a run of segments (one tile's units); a
// segment that holds all of its tile's units writes `out`, any other one (at
// most the first and the last of a range) writes a piece: the unnormalised
// accumulator with its running maximum (log2 units) and sum.
// prefill_merge_kernel folds the pieces of every cut tile in CTA order, so
// the same call gives the same bits every time.
#pragma once

#include <type_traits>

#include "decode_merge.cuh"  // store_out
#include "pa_internal.h"

namespace pa {

// One tile of the list.
struct PrefillTile {
    int32_t seq;   // sequence (block-table row)
    int32_t row0;  // row of q / out of its first token
    int32_t ntok;  // tokens in this tile
    int32_t p0;    // position of its first token (negative: before the sequence's first key)
};

// Where a CTA's walk over its range starts (one read of 80 bytes instead of a
// chain of dependent ones).
struct __align__(16) WalkStart {
    PrefillTile t, t_next;           // the first tile and the one after it
    int64_t x, hi;                   // weight position of the tile's start, end of the range
    int32_t kvh, k, j0, j1;
    int32_t nu, tiles, w_next, work; // work: 0 for a CTA without units
};

// A tile cut between CTAs, for the merge: pieces slot0 (of CTA
// slot0 / 2, its first units), then the first slots of the CTAs up to c1.
struct __align__(16) MergeEntry {
    int32_t row0, rows;  // the tile's first row of q / out, its query rows
    int32_t kvh, slot0, c1;
    int32_t pad[3];
};

// The call, as its kernels see it (one struct, passed by value).
struct PrefillArgs {
    const void *q;
    void *out;
    const void *k_cache, *v_cache;
    const uint8_t *k_scale, *v_scale;  // 8-bit caches: biased scale exponents [NB, B, Hk]
    const int32_t *tables, *seq_lens;
    const int32_t *cu_q;  // nullptr: one new token per sequence
    int32_t max_blocks, N, T, H, Hk, G, NB, B;  // (pa_decode_fp8's tensor-core kernel: Hk head groups of G query heads)
    int32_t tq1;          // tokens per row tile of the kernel (rows / G)
    int32_t rows;         // query rows of one row tile
    int32_t nrt;          // row tiles per tile (tq = tq1 * nrt)
    int32_t kt;           // keys per unit
    int32_t extra;        // weight of a tile beside its units
    int32_t C;            // persistent CTAs
    int32_t max_tiles;    // capacity of tiles[] and cu[]
    float scale_log2;
    int32_t few;          // 1: few tiles in many pieces, merged by prefill_merge_few_kernel
    int32_t *ctl;         // ctl[1]: cut tiles listed, ctl[2]: most query rows of one
    MergeEntry *merges;   // [C] the cut tiles (note_cut)
    int32_t *seq_tile0;   // [N + 1] first tile of each sequence
    int32_t *cu;          // [max_tiles + 1] exclusive prefix sums of the tiles' weights
    PrefillTile *tiles;   // [max_tiles]
    WalkStart *starts;    // [C]
    float2 *ml;           // [2 C][nrt * rows]
    float *acc;           // [2 C][nrt * rows][D]
    unsigned int *err;
    unsigned long long wait_ns;  // limit of the tcgen05 kernel's longest waits
};

__device__ __forceinline__ int32_t prefill_units(const PrefillTile &t, int32_t kt) {
    const int32_t keys = t.p0 + t.ntok;
    return keys <= kt ? 1 : (int32_t)(((int64_t)keys + kt - 1) / kt);  // no key: one unit that writes zeros
}

// Inclusive block-wide scan of x over 1024 threads plus carry; returns this
// thread's inclusive sum, *total the sum with the carry.
__device__ __forceinline__ int32_t block_scan_1024(int32_t x, int32_t carry, int32_t *warp_incl, int32_t *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous scan's reads of warp_incl
    if (lane == 31) warp_incl[w] = x;
    __syncthreads();
    if (w == 0) {
        int32_t s = warp_incl[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_incl[lane] = s;
    }
    __syncthreads();
    *total = carry + warp_incl[31];
    return carry + x + (w > 0 ? warp_incl[w - 1] : 0);
}

// Largest i in [0, n) with cu[i] <= x (cu not decreasing, cu[0] <= x).
__device__ __forceinline__ int32_t last_at_most(const int32_t *cu, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// One CTA: the tiles of every sequence, the prefix sums of their units, and
// the tile in which each CTA's range starts.  Row offsets that are not
// increasing within [0, T] void the whole call (no tile: out stays as it
// was), a length outside the table's reach counts as 0; both are recorded.
static __global__ void __launch_bounds__(1024) prefill_plan_kernel(const PrefillArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int32_t kSmemCu = 8192, kSmemSeqs = 2048;
    __shared__ int32_t warp_incl[32];
    __shared__ int32_t cu_s[kSmemCu], tile0_s[kSmemSeqs];
    const int tid = threadIdx.x;
    const int64_t max_len = (int64_t)a.max_blocks * a.B;
    const int32_t tq = a.tq1 * a.nrt;
    bool ok = true;
    if (a.cu_q) {
        for (int32_t i = tid; i <= a.N; i += 1024) {
            const int32_t x = a.cu_q[i];
            ok = ok && x >= 0 && x <= a.T && (i == 0 || a.cu_q[i - 1] <= x);
        }
    }
    ok = __syncthreads_and(ok) != 0;
    if (!ok) {
        if (tid == 0) {
            atomicOr(a.err, kErrBounds);
            a.ctl[1] = a.ctl[2] = 0;
            a.cu[0] = 0;
        }
        for (int32_t c = tid; c < a.C; c += 1024) a.starts[c] = WalkStart{};  // no work
        return;
    }
    int32_t *tile0 = a.N <= kSmemSeqs ? tile0_s : a.seq_tile0;  // first tile of each sequence
    int32_t tiles = 0;
    for (int32_t base = 0; base < a.N; base += 1024) {
        const int32_t i = base + tid;
        int32_t nt = 0;
        if (i < a.N) {
            const int32_t n = a.cu_q ? a.cu_q[i + 1] - a.cu_q[i] : 1;
            nt = (int32_t)(((int64_t)n + tq - 1) / tq);
            const int32_t L = a.seq_lens[i];
            if (L < 0 || L > max_len) atomicOr(a.err, kErrLength);
        }
        int32_t total;
        const int32_t incl = block_scan_1024(nt, tiles, warp_incl, &total);
        if (i < a.N) tile0[i] = incl - nt;
        tiles = total;
    }
    __syncthreads();  // tile0 is read by this CTA's other threads
    const bool in_smem = tiles + 1 <= kSmemCu;
    int32_t units = 0;
    for (int32_t base = 0; base < tiles; base += 1024) {
        const int32_t k = base + tid;
        int32_t u = 0;
        if (k < tiles) {
            // the last sequence that starts at or before tile k (it has tiles);
            // single queries: a tile each
            const int32_t lo = a.cu_q ? last_at_most(tile0, a.N, k) : k;
            const int32_t r0 = a.cu_q ? a.cu_q[lo] : lo, n = a.cu_q ? a.cu_q[lo + 1] - r0 : 1;
            const int32_t t0 = (k - tile0[lo]) * tq;
            int32_t L = a.seq_lens[lo];
            if (L < 0 || L > max_len) L = 0;
            PrefillTile t;
            t.seq = lo;
            t.row0 = r0 + t0;
            t.ntok = min(tq, n - t0);
            t.p0 = L - n + t0;
            a.tiles[k] = t;
            u = prefill_units(t, a.kt) + a.extra;
        }
        int32_t total;
        const int32_t incl = block_scan_1024(u, units, warp_incl, &total);
        if (k < tiles) {
            a.cu[k] = incl - u;
            if (in_smem) cu_s[k] = incl - u;
        }
        units = total;
    }
    if (tid == 0) {
        a.cu[tiles] = units;
        a.ctl[1] = a.ctl[2] = 0;
    }
    __syncthreads();
    const int32_t *cu = in_smem ? cu_s : a.cu;
    const int64_t W = (int64_t)a.Hk * units;
    const int32_t Ce = (int32_t)min(W, (int64_t)a.C);
    for (int32_t c = tid; c < a.C; c += 1024) {
        WalkStart w{};
        if (c < Ce) {
            const int64_t lo = split_begin(c, W, Ce);
            w.hi = split_begin((int64_t)c + 1, W, Ce);
            w.kvh = (int32_t)(lo / units);
            const int32_t r = (int32_t)(lo - (int64_t)w.kvh * units);
            w.k = last_at_most(cu, tiles, r);
            w.tiles = tiles;
            const int32_t begin = cu[w.k], next = w.k + 1 == tiles ? 0 : w.k + 1;
            auto end_of = [&](int32_t k) { return k + 1 == tiles ? units : cu[k + 1]; };
            w.t = a.tiles[w.k];
            w.t_next = a.tiles[next];
            w.x = lo - (r - begin);
            w.nu = end_of(w.k) - begin - a.extra;
            w.w_next = end_of(next) - cu[next];
            w.j0 = max(0, r - begin - a.extra);
            w.j1 = (int32_t)max((int64_t)0, min((int64_t)w.nu, w.hi - w.x - a.extra));
            w.work = w.j1 > w.j0 ? 1 : 0;
        }
        a.starts[c] = w;
    }
}

// A CTA's walk over its range: segments of consecutive units of one tile.
// kAhead: the next tile is read a segment ahead, so that moving on waits for no
// load (at the price of five registers).
template <bool kAhead>
struct PrefillWalk {
    int64_t x, hi;     // weight position of the current tile's start, end of the range
    int32_t kvh, k;    // KV head and tile of the current segment
    int32_t j0, j1;    // its units [j0, j1)
    int32_t nu;        // units of its tile
    int32_t tiles;
    bool first;        // the range's first segment
    PrefillTile t;     // the tile
    PrefillTile t_next;
    int32_t w_next;    // weight of the next tile

    // False when the CTA has no work.
    __device__ __forceinline__ bool init(const PrefillArgs &a, int32_t c) {
        const WalkStart w = a.starts[c];
        x = w.x, hi = w.hi, kvh = w.kvh, k = w.k, j0 = w.j0, j1 = w.j1, nu = w.nu, tiles = w.tiles;
        first = true;
        t = w.t, t_next = w.t_next, w_next = w.w_next;
        return w.work != 0;
    }
    __device__ __forceinline__ int32_t units_to_end(const PrefillArgs &a) const {
        return (int32_t)max((int64_t)0, min((int64_t)nu, hi - x - a.extra));
    }
    __device__ __forceinline__ void read_next(const PrefillArgs &a) {
        const int32_t n = k + 1 == tiles ? 0 : k + 1;
        t_next = a.tiles[n];
        w_next = a.cu[n + 1] - a.cu[n];
    }
    // Moves to the next segment; false at the range's end.
    __device__ __forceinline__ bool next(const PrefillArgs &a) {
        x += nu + a.extra;
        first = false;
        if (++k == tiles) {
            k = 0;
            ++kvh;
        }
        if constexpr (kAhead) {
            t = t_next;
            nu = w_next - a.extra;
        } else {
            t = a.tiles[k];
            nu = a.cu[k + 1] - a.cu[k] - a.extra;
        }
        j0 = 0;
        j1 = units_to_end(a);
        if (j1 == 0) return false;
        if constexpr (kAhead) read_next(a);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == nu; }
    // Slot of this segment's piece: a range has at most two, its first segment's and its last one's.
    __device__ __forceinline__ int64_t slot(int32_t c) const { return 2 * (int64_t)c + (first ? 0 : 1); }
};
using PrefillCursor = PrefillWalk<true>;

// CTA c, by one thread: the tile that its range's start cuts between units,
// for the merge, if CTA c - 1 holds that tile's first unit (so each cut tile
// once).  With few tiles (a.few) the entries form a list; else entry c stands
// at c, with no rows where there is nothing to merge.
template <class Walk>
__device__ __forceinline__ void note_cut(const PrefillArgs &a, int32_t c, bool work, const Walk &cur) {
    MergeEntry me{};
    if (work && cur.j0 > 0) {
        const int64_t W = (int64_t)a.Hk * a.cu[cur.tiles];
        const int32_t Ce = (int32_t)min(W, (int64_t)a.C);
        const int32_t c0 = split_owner(cur.x + a.extra, W, Ce);
        if (c0 == c - 1) {
            me.row0 = cur.t.row0;
            me.rows = cur.t.ntok * a.G;
            me.kvh = cur.kvh;
            me.slot0 = 2 * c0 + (split_begin(c0, W, Ce) >= cur.x ? 0 : 1);
            me.c1 = split_owner(cur.x + a.extra + cur.nu - 1, W, Ce);
        }
    }
    if (!a.few) {
        a.merges[c] = me;
    } else if (me.rows > 0) {
        a.merges[atomicAdd(a.ctl + 1, 1)] = me;
        atomicMax(a.ctl + 2, me.rows);
    }
}

// Merge of the listed tiles, few of them in many pieces each: a block takes 8
// query rows of one, a warp per row, its lanes across the columns, kBatch
// pieces in flight, folded in CTA order.  16 long contexts cut in 19 pieces
// each: 8 us, where the kernel below, a block per CTA boundary and quarter of
// the rows, most of them without work, took 16 to 20; with hundreds of tiles
// cut in two or three pieces that one is the faster (its blocks find their
// tile without a list).
constexpr int kMergeWarps = 8, kMergeCtas = 4;  // per block, blocks per SM
template <typename T, int D>
static __global__ void __launch_bounds__(32 * kMergeWarps)
    prefill_merge_few_kernel(const __grid_constant__ PrefillArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int E = D / 32, NV = E == 8 ? 2 : 1, NE = E / NV;  // accumulator elements of a lane, vectors, elements of one
    constexpr int kBatch = D == 256 ? 4 : 8;
    using Vec = typename std::conditional<NE == 2, float2, float4>::type;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slot_rows = (int64_t)a.nrt * a.rows;
    const int32_t cuts = a.ctl[1], chunks = (a.ctl[2] + kMergeWarps - 1) / kMergeWarps;
    for (int32_t item = blockIdx.x; item < cuts * chunks; item += gridDim.x) {
        const MergeEntry me = a.merges[item % cuts];
        const int32_t i = item / cuts * kMergeWarps + warp;  // query row of the tile
        if (i >= me.rows) continue;
        const int32_t tok = i / a.G, g = i - tok * a.G;
        const int64_t row = (int64_t)(tok / a.tq1) * a.rows + (tok % a.tq1) * a.G + g;
        const int32_t c0 = me.slot0 >> 1, np_all = me.c1 - c0 + 1;
        auto piece = [&](int32_t p) {  // row of the p-th piece
            return (p == 0 ? (int64_t)me.slot0 : 2 * (int64_t)(c0 + p)) * slot_rows + row;
        };
        float M = -INFINITY, l = 0.f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int32_t p0 = 0; p0 < np_all; p0 += 32) {
            const int32_t np = min(32, np_all - p0);
            // 32 pieces' statistics, one per lane, with the first accumulators in flight
            float2 v = make_float2(-INFINITY, 0.f);
            if (lane < np) v = __ldcg(&a.ml[piece(p0 + lane)]);
            float wgt = 0.f;
            for (int32_t b0 = 0; b0 < np; b0 += kBatch) {
                Vec x[kBatch][NV];
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (b0 + b < np) {
                        const Vec *ap = reinterpret_cast<const Vec *>(a.acc + piece(p0 + b0 + b) * D + lane * E);
#pragma unroll
                        for (int e = 0; e < NV; ++e) x[b][e] = __ldcg(ap + e);
                    }
                if (b0 == 0) {
                    float mb = v.x;
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, s));
                    const float Mn = fmaxf(M, mb), mref = Mn == -INFINITY ? 0.f : Mn;  // no key so far: zeros
                    const float sc = ex2_approx(M - mref);
                    wgt = ex2_approx(v.x - mref);
                    float lw = wgt * v.y;
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, s);
                    l = l * sc + lw;
                    M = Mn;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] *= sc;
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const float w = __shfl_sync(0xffffffffu, wgt, (b0 + b) & 31);
                    if (b0 + b < np) {
#pragma unroll
                        for (int e = 0; e < NV; ++e) {
                            const float *xe = reinterpret_cast<const float *>(&x[b][e]);
#pragma unroll
                            for (int q = 0; q < NE; ++q) o[e * NE + q] = fmaf(w, xe[q], o[e * NE + q]);
                        }
                    }
                }
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a row without keys is zero
        T *op = (T *)a.out + ((int64_t)(me.row0 + tok) * a.H + (int64_t)me.kvh * a.G + g) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {  // out is aligned to two elements
            if constexpr (std::is_same<T, float>::value)
                *reinterpret_cast<float2 *>(op + e) = make_float2(o[e] * inv, o[e + 1] * inv);
            else
                *reinterpret_cast<uint32_t *>(op + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
        }
    }
}

// Merge of the cut tiles, many of them in a few pieces each: block (c - 1, y)
// takes its share of the rows of entry c.  A warp folds two rows at once, its
// lanes across the columns, up to four pieces of each in flight, in CTA order;
// bound by the latency of two dependent reads through L2 (the entry, the
// pieces).  150 tiles of 256 rows in two or three pieces (45 MB): 12 to 14 us,
// against 22 us with a row at a time behind a search of the work list.
template <typename T, int D>
static __global__ void __launch_bounds__(32 * kMergeWarps, D == 256 ? 2 : 4)
    prefill_merge_kernel(const __grid_constant__ PrefillArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int E = D / 32, NV = E == 8 ? 2 : 1, NE = E / NV;  // accumulator elements of a lane, vectors, elements of one
    constexpr int kRows = 2, kBatch = 4;
    using Vec = typename std::conditional<NE == 2, float2, float4>::type;
    const MergeEntry me = a.merges[blockIdx.x + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slot_rows = (int64_t)a.nrt * a.rows;
    const int32_t c0 = me.slot0 >> 1, np = me.c1 - c0 + 1, stride = gridDim.y * kMergeWarps;
    auto piece = [&](int32_t p) { return (p == 0 ? (int64_t)me.slot0 : 2 * (int64_t)(c0 + p)) * slot_rows; };
    for (int32_t i0 = blockIdx.y * kMergeWarps + warp; i0 < me.rows; i0 += kRows * stride) {
        int64_t row[kRows];
        float M[kRows], l[kRows], o[kRows][E];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int32_t i = min(i0 + r * stride, me.rows - 1), tok = i / a.G;
            row[r] = (int64_t)(tok / a.tq1) * a.rows + (tok % a.tq1) * a.G + (i - tok * a.G);
            M[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[r][e] = 0.f;
        }
        for (int32_t p0 = 0; p0 < np; p0 += kBatch) {
            Vec x[kRows][kBatch][NV];
            float2 v[kRows][kBatch];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    v[r][b] = make_float2(-INFINITY, 0.f);
                    if (p0 + b < np) {
                        const int64_t at = piece(p0 + b) + row[r];
                        v[r][b] = __ldcg(&a.ml[at]);
                        const Vec *ap = reinterpret_cast<const Vec *>(a.acc + at * D + lane * E);
#pragma unroll
                        for (int e = 0; e < NV; ++e) x[r][b][e] = __ldcg(ap + e);
                    }
                }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float Mn = M[r];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) Mn = fmaxf(Mn, v[r][b].x);
                const float mref = Mn == -INFINITY ? 0.f : Mn;  // no key so far: zeros
                const float sc = ex2_approx(M[r] - mref);
                M[r] = Mn;
                l[r] *= sc;
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] *= sc;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    if (p0 + b >= np) break;
                    const float w = ex2_approx(v[r][b].x - mref);
                    l[r] = fmaf(w, v[r][b].y, l[r]);
#pragma unroll
                    for (int e = 0; e < NV; ++e) {
                        const float *xe = reinterpret_cast<const float *>(&x[r][b][e]);
#pragma unroll
                        for (int q = 0; q < NE; ++q) o[r][e * NE + q] = fmaf(w, xe[q], o[r][e * NE + q]);
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int32_t i = i0 + r * stride;
            if (i >= me.rows) break;
            const int32_t tok = i / a.G, g = i - tok * a.G;
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];  // a row without keys is zero
            T *op = (T *)a.out + ((int64_t)(me.row0 + tok) * a.H + (int64_t)me.kvh * a.G + g) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {  // out is aligned to two elements
                if constexpr (std::is_same<T, float>::value)
                    *reinterpret_cast<float2 *>(op + e) = make_float2(o[r][e] * inv, o[r][e + 1] * inv);
                else
                    *reinterpret_cast<uint32_t *>(op + e) = pack_bf16x2(o[r][e] * inv, o[r][e + 1] * inv);
            }
        }
    }
}

}  // namespace pa
