// Write into the 8-bit cache with block scales (pa_write_blocks_fp8).
//
// A block and KV head share one exponent: e = max over the call's rows in that
// block of the row exponent (fp8_codec.cuh), and at least the e that the block
// has where it holds earlier positions; codes are e4m3(x 2^-e).  So the unit of
// work is (sequence, block it touches, KV head): a team of W warps loads the
// unit's rows of K and V once (16-byte vectors, up to kVecs of each a thread, all
// in flight together), reduces the largest |x|, and encodes what it still holds
// in registers.  No unit shares a block with another, so there are no atomics and
// the result does not depend on any order.  A unit's rows are Hk * D elements
// apart, D contiguous ones each.
//
// The units are not listed anywhere: sequence i's are numbered from
// cu_q_lens[i] / B + 2 i, which leaves room for the floor((n - 2) / B) + 2 blocks
// that n tokens can touch, so a team finds its sequence by a search in the
// offsets (in shared memory) and some numbers stand for nothing.
//
// Bound by HBM traffic (x once, codes once) on prompts and by latency on a
// decode step.
#include "fp8_rows.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kVecs = 8;             // vectors of K, and of V, that a thread holds
constexpr int kWriteBlocksCtas = 2;  // resident CTAs per SM that its registers are held to
constexpr int kCuSmem = 2048;     // offsets kept in shared memory
constexpr int kByteMax = kScaleMax + kScaleBias;  // largest byte that a write makes

struct WriteBlocksArgs {
    const void *k, *v;
    const int32_t *tables, *seq_lens, *cu;
    int32_t max_blocks, N, T;
    uint8_t *kc, *vc, *ks, *vs;
    int32_t NB, B, Hk, D;
    uint32_t units;  // numbers of units, of which each has Hk items
    unsigned int *err;
};

// One unit: the block, its first and last new row.
struct WriteUnit {
    int32_t phys;   // -1: nothing to do
    int32_t off;    // first position of the block that the call writes
    int32_t row0;   // row of k and v that goes there
    int32_t ntok;
    int32_t held;   // positions of the block that the sequence held before: 0 or off
};

__device__ __forceinline__ int32_t unit_base(int32_t cu, int32_t i, int32_t B) { return cu / B + 2 * i; }

// cu: the offsets (checked: not decreasing, within [0, T]).
__device__ __forceinline__ WriteUnit find_unit(const WriteBlocksArgs &a, const int32_t *cu, uint32_t u) {
    WriteUnit w{-1, 0, 0, 0, 0};
    int32_t lo = 0, hi = a.N - 1;  // the last sequence whose numbers begin at or before u
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if ((uint32_t)unit_base(cu[mid], mid, a.B) <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int32_t c0 = cu[lo], n = cu[lo + 1] - c0;
    const int32_t base = unit_base(c0, lo, a.B);
    if (n == 0 || u < (uint32_t)base) return w;
    const int32_t L = a.seq_lens[lo];
    if (L < n || L > (int64_t)a.max_blocks * a.B) {
        if (u == (uint32_t)base) atomicOr(a.err, kErrLength);
        return w;
    }
    // The spare numbers (and those of a padded batch's rows) are told by their
    // distance: the block itself may lie past 32 bits.
    const int32_t start = L - n, first = start / a.B;
    const uint32_t at = u - (uint32_t)base;
    if (at > (uint32_t)((L - 1) / a.B - first)) return w;
    const int32_t blk = first + (int32_t)at;
    const int32_t p0 = max(start, blk * a.B);  // first new position of the block
    w.off = p0 - blk * a.B;
    w.held = w.off;
    w.row0 = c0 + (p0 - start);
    w.ntok = min(L - p0, a.B - w.off);
    const int32_t b = a.tables[(int64_t)lo * a.max_blocks + blk];
    if (b < 0 || b >= a.NB)
        atomicOr(a.err, kErrBounds);
    else
        w.phys = b;
    return w;
}

// The offsets into shared memory where they fit; false if they are not in order.
__device__ __forceinline__ bool load_offsets(const WriteBlocksArgs &a, int32_t *cu_s) {
    bool ok = true;
    for (int32_t i = threadIdx.x; i <= a.N; i += blockDim.x) {
        const int32_t x = a.cu[i];
        ok = ok && x >= 0 && x <= a.T && (i == 0 || a.cu[i - 1] <= x);
        if (i < kCuSmem) cu_s[i] = x;
    }
    ok = __syncthreads_and(ok) != 0;
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrBounds);
    return ok;
}

// Exponent of a block from the call's largest |x| and the byte that it has, and
// the byte that it gets.
__device__ __forceinline__ int32_t block_exponent(uint32_t amax, int32_t held, uint32_t old, uint32_t *byte) {
    int32_t e = row_exponent(amax);
    *byte = (uint32_t)(e + kScaleBias);
    if (held > 0) {
        e = max(e, (int32_t)min(old, (uint32_t)kByteMax) - kScaleBias);
        *byte = old > kByteMax ? old : (uint32_t)(e + kScaleBias);
    }
    return e;
}
// Factor of the codes that a block holds when its exponent grows to e (below
// 2^-126 every code becomes 0 anyway), 1 when it stays.
__device__ __forceinline__ float recode_factor(int32_t e, uint32_t old) {
    const int32_t d = e - ((int32_t)min(old, (uint32_t)kByteMax) - kScaleBias);
    return d > 0 ? inv_scale(min(d, 126)) : 1.f;
}

template <int W>
__device__ __forceinline__ void team_sync(int team) {
    if constexpr (W == 1)
        __syncwarp();
    else if constexpr (W == 8)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * W) : "memory");
}

// Codes that a block holds from before (rows [0, held) of one head), recoded by f;
// members of a team of n threads.
__device__ __forceinline__ void recode_rows(uint8_t *codes, int32_t held, int32_t D, int64_t stride, float f, uint32_t ti,
                                            uint32_t n) {
    const uint32_t wr = (uint32_t)D / 4;
    for (uint32_t i = ti; i < (uint32_t)held * wr; i += n) {
        const uint32_t row = i / wr;
        uint32_t *p = reinterpret_cast<uint32_t *>(codes + (int64_t)row * stride) + (i - row * wr);
        const float4 y = decode4(*p);
        *p = encode4(y.x * f, y.y * f, y.z * f, y.w * f);
    }
}

// Rows of whole 16-byte vectors, as many per row (vecs) as divide the team and as
// many per block as its registers hold: a team of W of the CTA's 8 warps takes a
// unit and `heads` of its KV heads, one after the other, K and V together.  A
// thread's vectors are the same column of rows a step apart.
// 48 prompts of 700 to 4500 tokens (8 heads, head_dim 128, bf16; 591 MB): 109 us, 5.4
// TB/s, 0.80 of the copy bandwidth (104 in a graph); fp32 (985 MB) 214 us, 4.6 TB/s;
// head_dim 64 75 and 109 us.  With a search per head and a division per vector it
// took 152 instructions per vector of 8 values and 161 us, when this form took 107; with
// half the vectors per thread and 3 or 4 CTAs 109 and 113 us.  One token of 64
// sequences: 4.3 to 4.4 us.
template <typename T, int W>
__global__ void __launch_bounds__(256, kWriteBlocksCtas) write_blocks_kernel(const __grid_constant__ WriteBlocksArgs a, const int32_t heads) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int N = Vec16<T>::N, kTeam = 32 * W, kTeams = 8 / W;
    __shared__ int32_t cu_s[kCuSmem];
    __shared__ uint32_t tops[2][8];
    if (!load_offsets(a, cu_s)) return;
    const int32_t *cu = a.N < kCuSmem ? cu_s : a.cu;
    const int team = threadIdx.x / kTeam, ti = threadIdx.x % kTeam, warp = threadIdx.x >> 5;
    const uint32_t Hk = (uint32_t)a.Hk, vecs = (uint32_t)a.D / N, stride = Hk * vecs;  // of a row, and from row to row
    const int32_t my_row = ti / (int32_t)vecs, rows_step = kTeam / (int32_t)vecs;
    const uint32_t my_at = (uint32_t)my_row * stride + ((uint32_t)ti - (uint32_t)my_row * vecs), step = (uint32_t)rows_step * stride;
    const uint32_t groups = (Hk + (uint32_t)heads - 1) / (uint32_t)heads;
    const uint64_t items = (uint64_t)a.units * groups;
    for (uint64_t item = (uint64_t)blockIdx.x * kTeams + team; item < items; item += (uint64_t)gridDim.x * kTeams) {
        const uint32_t u = (uint32_t)(item / groups), h0 = (uint32_t)(item - (uint64_t)u * groups) * (uint32_t)heads;
        const WriteUnit w = find_unit(a, cu, u);
        if (w.phys < 0) continue;  // the same for the whole team
        const int64_t from = (int64_t)w.row0 * stride + h0 * vecs + my_at;
        const uint4 *src[2] = {reinterpret_cast<const uint4 *>(a.k) + from, reinterpret_cast<const uint4 *>(a.v) + from};
        const int64_t to = (((int64_t)w.phys * a.B + w.off) * stride + h0 * vecs + my_at) * N;
        uint8_t *dst[2] = {a.kc + to, a.vc + to};
        const int64_t sc = (int64_t)w.phys * Hk + h0;
        const int32_t left = w.ntok - my_row;  // this thread's rows: j * rows_step < left
        const uint32_t h1 = min(h0 + (uint32_t)heads, Hk);
        for (uint32_t h = h0; h < h1; ++h) {
            uint8_t *scale[2] = {a.ks + sc + (h - h0), a.vs + sc + (h - h0)};
            uint32_t old[2] = {0u, 0u};
            if (w.held > 0) old[0] = *scale[0], old[1] = *scale[1];
            uint4 r[2][kVecs];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < kVecs; ++j)
                    r[s][j] = j * rows_step < left ? __ldcs(src[s] + j * step) : make_uint4(0u, 0u, 0u, 0u);
            uint32_t top[2] = {0u, 0u};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int j = 0; j < kVecs; ++j) top[s] = max(top[s], Vec16<T>::largest(r[s][j]));
                top[s] = __reduce_max_sync(0xffffffffu, top[s]);
            }
            if constexpr (W > 1) {
                if ((threadIdx.x & 31) == 0) tops[0][warp] = top[0], tops[1][warp] = top[1];
                team_sync<W>(team);
#pragma unroll
                for (int k = 0; k < W; ++k) top[0] = max(top[0], tops[0][team * W + k]), top[1] = max(top[1], tops[1][team * W + k]);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                uint32_t byte;
                const int32_t e = block_exponent(Vec16<T>::bits(top[s]), w.held, old[s], &byte);
                const float inv = inv_scale(e);
#pragma unroll
                for (int j = 0; j < kVecs; ++j)
                    if (j * rows_step < left) {
                        float f[N];
                        Vec16<T>::load(r[s][j], f);
                        store_codes<N>(dst[s] + (uint64_t)j * step * N, f, inv);
                    }
                if (w.held > 0) {
                    const float f = recode_factor(e, old[s]);
                    if (f != 1.f)
                        recode_rows((s ? a.vc : a.kc) + ((int64_t)w.phys * a.B * Hk + h) * a.D, w.held, a.D, (int64_t)Hk * a.D, f, ti, kTeam);
                }
                old[s] = byte;
            }
            team_sync<W>(team);  // the old bytes and tops have been read
            if (ti < 2) *(ti ? scale[1] : scale[0]) = (uint8_t)(ti ? old[1] : old[0]);  // (an index would put both in memory)
            src[0] += vecs, src[1] += vecs;
            dst[0] += a.D, dst[1] += a.D;
        }
    }
}

// Any row length and alignment: a warp per item, an element per lane at a time,
// two passes over the rows (the second finds them in L1 or L2).
template <typename T>
__global__ void __launch_bounds__(256) write_blocks_any_kernel(const __grid_constant__ WriteBlocksArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ int32_t cu_s[kCuSmem];
    if (!load_offsets(a, cu_s)) return;
    const int32_t *cu = a.N < kCuSmem ? cu_s : a.cu;
    const int lane = threadIdx.x & 31;
    const uint32_t Hk = (uint32_t)a.Hk, D = (uint32_t)a.D;  // 2 Hk and D + 31 may pass 2^31
    const uint64_t items = (uint64_t)a.units * (2 * Hk);
    for (uint64_t item = ((uint64_t)blockIdx.x * 256 + threadIdx.x) >> 5; item < items; item += (uint64_t)gridDim.x * 8) {
        const uint32_t u = (uint32_t)(item / (2 * Hk)), hs = (uint32_t)(item - (uint64_t)u * (2 * Hk));
        const bool is_v = hs >= Hk;
        const uint32_t h = is_v ? hs - Hk : hs;
        const WriteUnit w = find_unit(a, cu, u);
        if (w.phys < 0) continue;
        const T *x = (const T *)(is_v ? a.v : a.k) + ((int64_t)w.row0 * a.Hk + h) * a.D;
        uint8_t *codes = (is_v ? a.vc : a.kc) + ((int64_t)w.phys * a.B * a.Hk + h) * a.D;  // of the block's first row
        uint8_t *scale = (is_v ? a.vs : a.ks) + (int64_t)w.phys * a.Hk + h;
        const int64_t stride = (int64_t)a.Hk * a.D;
        const uint32_t old = w.held > 0 ? *scale : 0u;
        uint32_t top = 0;
        for (int32_t t = 0; t < w.ntok; ++t)
            for (uint32_t d = lane; d < D; d += 32) top = max(top, finite_bits(to_f32(x[t * stride + d])));
        top = __reduce_max_sync(0xffffffffu, top);
        uint32_t byte;
        const int32_t e = block_exponent(top, w.held, old, &byte);
        const float inv = inv_scale(e), f = recode_factor(e, old);
        for (int32_t t = 0; t < w.ntok; ++t)
            for (uint32_t d = lane; d < D; d += 32)
                codes[(w.off + t) * stride + d] =
                    (uint8_t)__nv_cvt_float_to_fp8(to_f32(x[t * stride + d]) * inv, __NV_SATFINITE, __NV_E4M3);
        if (w.held > 0 && f != 1.f)
            for (int32_t t = 0; t < w.held; ++t)
                for (uint32_t d = lane; d < D; d += 32) {
                    uint8_t *p = codes + t * stride + d;
                    *p = (uint8_t)__nv_cvt_float_to_fp8(decode4(*p).x * f, __NV_SATFINITE, __NV_E4M3);
                }
        __syncwarp();
        if (lane == 0) *scale = (uint8_t)byte;
    }
}

namespace {

template <typename T>
cudaError_t launch_write_blocks(const WriteBlocksArgs &a, cudaStream_t s) {
    WriteBlocksArgs arg = a;
    const int64_t vecs = a.D / Vec16<T>::N, block_vecs = vecs * a.B;  // of a row, of a block and head
    int W = 1;  // as few warps as hold a block and head
    while (W < 8 && block_vecs > 32 * kVecs * W) W *= 2;
    if (!aligned_rows<T>(a.D, a.k, a.v, a.kc, a.vc) || block_vecs > 32 * kVecs * W || 32 * W % vecs != 0 ||
        block_vecs * a.Hk >= ((int64_t)1 << 28)) {
        void *args[] = {&arg};
        const int64_t items = (int64_t)a.units * 2 * a.Hk;
        return launch_pdl((const void *)write_blocks_any_kernel<T>, dim3(grid_for((items + 7) / 8, 8)), dim3(256), args, 0, s);
    }
    const void *fn = W == 1   ? (const void *)write_blocks_kernel<T, 1>
                     : W == 2 ? (const void *)write_blocks_kernel<T, 2>
                     : W == 4 ? (const void *)write_blocks_kernel<T, 4>
                              : (const void *)write_blocks_kernel<T, 8>;
    // All heads of a unit by one team where that still fills the GPU, else one.
    const int64_t teams = (int64_t)std::max(num_sms(), 1) * kWriteBlocksCtas * (8 / W);
    int32_t heads = (int64_t)a.units >= 2 * teams ? a.Hk : 1;
    const int64_t items = (int64_t)a.units * ((a.Hk + heads - 1) / heads);
    void *args[] = {&arg, &heads};
    return launch_pdl(fn, dim3(grid_for((items * W + 7) / 8, kWriteBlocksCtas)), dim3(256), args, 0, s);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status_t pa_write_blocks_fp8(const void *k, const void *v, int32_t dtype, const int32_t *block_tables,
                                           int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *cu_q_lens,
                                           int32_t num_seqs, int32_t num_tokens, void *k_cache, void *v_cache,
                                           uint8_t *k_scale, uint8_t *v_scale, const pa_cache_desc_t *cache,
                                           pa_stream_t stream) try {
    const pa_status_t st = validate_fp8_desc(cache);
    if (st != PA_OK) return st;
    if (cache->dtype != PA_FP8_E4M3_BLOCK) return PA_ERR_INVALID_ARG;
    if (num_seqs < 0 || num_tokens < 0 || (dtype != PA_F32 && dtype != PA_BF16)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!k || !v || !block_tables || !seq_lens || !cu_q_lens || !k_cache || !v_cache || !k_scale || !v_scale)
        return PA_ERR_INVALID_ARG;
    if (max_blocks_per_seq <= 0 || (int64_t)num_seqs * max_blocks_per_seq >= ((int64_t)1 << 31) ||
        (int64_t)max_blocks_per_seq * cache->block_size >= ((int64_t)1 << 31))
        return PA_ERR_INVALID_ARG;
    if (((uintptr_t)k | (uintptr_t)v) % (size_t)dtype_bytes(dtype) != 0) return PA_ERR_INVALID_ARG;
    const int64_t units = (int64_t)num_tokens / cache->block_size + 2 * (int64_t)num_seqs;
    if (units >= ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;  // unit numbers are 32 bits
    WriteBlocksArgs a{};
    a.k = k;
    a.v = v;
    a.tables = block_tables;
    a.seq_lens = seq_lens;
    a.cu = cu_q_lens;
    a.max_blocks = max_blocks_per_seq;
    a.N = num_seqs;
    a.T = num_tokens;
    a.kc = (uint8_t *)k_cache;
    a.vc = (uint8_t *)v_cache;
    a.ks = k_scale;
    a.vs = v_scale;
    a.NB = cache->num_blocks;
    a.B = cache->block_size;
    a.Hk = cache->num_kv_heads;
    a.D = cache->head_dim;
    a.units = (uint32_t)units;
    a.err = device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    cudaGetLastError();
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == PA_BF16 ? launch_write_blocks<__nv_bfloat16>(a, s) : launch_write_blocks<float>(a, s);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
} catch (...) {
    return host_failure();
}
