// Chunk attention over the paged cache (pa_prefill): host side and the work
// list and merge kernels.  The attention kernels are prefill_tc.cuh (tcgen05)
// and prefill_simt.cuh (CUDA cores); prefill_plan.cuh describes the split.
#include <cmath>

#include "prefill_kernels.h"
#include "prefill_simt.cuh"
#include "prefill_tc.cuh"

namespace pa {

namespace {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

bool tc_supported(const pa_cache_desc_t *c, int G) {
    return c->dtype == PA_BF16 && c->layout == PA_LAYOUT_ROW && (c->head_dim == 64 || c->head_dim == 128) &&
           c->block_size % 8 == 0 && G <= 64;
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// Maps of the tcgen05 kernel: K and V as {64 elements, NB * B rows, D / 64
// panels, Hk heads} in boxes of gran rows of one panel and head; q as {64, D / 64
// panels, H, T} in boxes of tq1 tokens x G heads of one panel.  All boxes land
// as 128-byte lines with the 128-byte swizzle.
bool encode_tc_maps(CUtensorMap *q, CUtensorMap *k, CUtensorMap *v, const PrefillArgs &a, const pa_cache_desc_t *c,
                    int gran) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t D = c->head_dim, Hk = c->num_kv_heads;
    const cuuint32_t one[4] = {1, 1, 1, 1};
    auto enc = [&](CUtensorMap *m, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
                   const cuuint32_t *box) {
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t kd[4] = {64, (cuuint64_t)c->num_blocks * c->block_size, D / 64, Hk};
    const cuuint64_t ks[3] = {Hk * D * 2, 128, D * 2};
    const cuuint32_t kb[4] = {64, (cuuint32_t)gran, 1, 1};
    const cuuint64_t qd[4] = {64, D / 64, (cuuint64_t)a.H, (cuuint64_t)a.T};
    const cuuint64_t qs[3] = {128, D * 2, (cuuint64_t)a.H * D * 2};
    const cuuint32_t qb[4] = {64, 1, (cuuint32_t)a.G, (cuuint32_t)a.tq1};
    return enc(k, a.k_cache, kd, ks, kb) && enc(v, a.v_cache, kd, ks, kb) && enc(q, a.q, qd, qs, qb);
}

}  // namespace

pa_status_t prefill_layout(bool tc, const pa_cache_desc_t *c, int32_t N, int32_t T, int32_t H, int32_t num_splits,
                           PrefillPlan *p) {
    const int32_t G = H / c->num_kv_heads;
    const void *fn = tc ? prefill_tc_ptr(c->head_dim, &p->smem)
                        : prefill_simt_ptr(c->dtype, c->head_dim, c->layout, &p->smem);
    if (!fn) return PA_ERR_UNSUPPORTED;
    p->tc = tc;
    p->rows = tc ? kTcRows : kSimtRows;
    p->nrt = tc ? 2 : 1;
    p->kt = tc ? kTcKeys : kSimtKeys;
    p->extra = tc ? kTcExtra : kSimtExtra;
    p->threads = tc ? kTcThreads : kSimtThreads;
    p->tq1 = p->rows / G;
    const int64_t tq = (int64_t)p->tq1 * p->nrt;
    const int64_t tiles = (int64_t)N + T / tq;  // sum of ceil(n_i / tq)
    if (tiles >= ((int64_t)1 << 30)) return PA_ERR_UNSUPPORTED;
    p->max_tiles = (int32_t)tiles;
    p->C = num_splits;
    if (p->C == 0) p->C = default_ctas(fn, p->threads, p->smem);
    if (p->C <= 0) return PA_ERR_CUDA;
    prefill_workspace(p, N, c->head_dim);
    return PA_OK;
}

void prefill_workspace(PrefillPlan *p, int32_t N, int32_t head_dim) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    const size_t tiles = (size_t)p->max_tiles;
    p->off_ctl = take(256);
    p->off_tile0 = take(sizeof(int32_t) * ((size_t)N + 1));
    p->off_cu = take(sizeof(int32_t) * (tiles + 1));
    p->off_tiles = take(sizeof(PrefillTile) * std::max<size_t>(tiles, 1));
    p->off_start = take(sizeof(WalkStart) * (size_t)p->C);
    p->off_merges = take(sizeof(MergeEntry) * (size_t)p->C);
    const size_t slot_rows = 2 * (size_t)p->C * p->nrt * p->rows;
    p->off_ml = take(sizeof(float2) * slot_rows);
    p->off_acc = take(sizeof(float) * slot_rows * head_dim);
    p->total = off;
}

pa_status_t prefill_bind(const PrefillPlan &p, PrefillArgs *a, void *workspace) {
    uint8_t *ws = (uint8_t *)workspace;
    a->tq1 = p.tq1;
    a->rows = p.rows;
    a->nrt = p.nrt;
    a->kt = p.kt;
    a->extra = p.extra;
    a->C = p.C;
    a->max_tiles = p.max_tiles;
    a->ctl = (int32_t *)(ws + p.off_ctl);
    a->seq_tile0 = (int32_t *)(ws + p.off_tile0);
    a->cu = (int32_t *)(ws + p.off_cu);
    a->tiles = (PrefillTile *)(ws + p.off_tiles);
    a->starts = (WalkStart *)(ws + p.off_start);
    a->merges = (MergeEntry *)(ws + p.off_merges);
    a->few = (int64_t)p.max_tiles * a->Hk * 4 <= p.C ? 1 : 0;
    a->ml = (float2 *)(ws + p.off_ml);
    a->acc = (float *)(ws + p.off_acc);
    a->err = device_error_word();
    return a->err ? PA_OK : PA_ERR_CUDA;
}

pa_status_t prefill_launch_plan(PrefillArgs &a, cudaStream_t s) {
    void *args[] = {&a};
    return launch_pdl((const void *)prefill_plan_kernel, dim3(1), dim3(1024), args, 0, s) == cudaSuccess ? PA_OK
                                                                                                       : PA_ERR_CUDA;
}

pa_status_t prefill_launch_merge(PrefillArgs &a, bool f32, int32_t head_dim, cudaStream_t s) {
    // a single CTA cuts no tile, nor is one of a single unit ever cut
    if (a.C <= 1 || (int64_t)a.max_blocks * a.B <= a.kt) return PA_OK;
    const void *fn = head_dim == 64    ? (f32 ? (const void *)prefill_merge_kernel<float, 64>
                                              : (const void *)prefill_merge_kernel<__nv_bfloat16, 64>)
                     : head_dim == 128 ? (f32 ? (const void *)prefill_merge_kernel<float, 128>
                                              : (const void *)prefill_merge_kernel<__nv_bfloat16, 128>)
                                       : (f32 ? (const void *)prefill_merge_kernel<float, 256>
                                              : (const void *)prefill_merge_kernel<__nv_bfloat16, 256>);
    void *args[] = {&a};
    if (a.few) {
        const void *few = head_dim == 64    ? (f32 ? (const void *)prefill_merge_few_kernel<float, 64>
                                                   : (const void *)prefill_merge_few_kernel<__nv_bfloat16, 64>)
                          : head_dim == 128 ? (f32 ? (const void *)prefill_merge_few_kernel<float, 128>
                                                   : (const void *)prefill_merge_few_kernel<__nv_bfloat16, 128>)
                                            : (f32 ? (const void *)prefill_merge_few_kernel<float, 256>
                                                   : (const void *)prefill_merge_few_kernel<__nv_bfloat16, 256>);
        const int rows = a.tq1 * a.nrt * a.G;
        const int64_t items = (int64_t)a.max_tiles * a.Hk * ((rows + kMergeWarps - 1) / kMergeWarps);
        const int grid = (int)std::min<int64_t>(items, kMergeCtas * std::max(num_sms(), 1));
        return launch_pdl(few, dim3(grid), dim3(32 * kMergeWarps), args, 0, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    }
    // up to 8 blocks share the rows of a cut tile, 4 rows a warp
    const int y = std::min((a.tq1 * a.nrt * a.G + 2 * kMergeWarps - 1) / (2 * kMergeWarps), 8);
    return launch_pdl(fn, dim3(a.C - 1, y), dim3(32 * kMergeWarps), args, 0, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t prefill_launch(const PrefillPlan &p, const pa_cache_desc_t *c, PrefillArgs a, void *workspace,
                           cudaStream_t s) {
    a.Hk = c->num_kv_heads;
    a.G = a.H / a.Hk;
    a.NB = c->num_blocks;
    a.B = c->block_size;
    pa_status_t st = prefill_bind(p, &a, workspace);
    if (st != PA_OK) return st;
    cudaGetLastError();  // clear a stale launch error so the checks below are ours
    if ((st = prefill_launch_plan(a, s)) != PA_OK) return st;
    void *args[] = {&a};
    size_t smem;
    const void *fn = p.tc ? prefill_tc_ptr(c->head_dim, &smem)
                          : prefill_simt_ptr(c->dtype, c->head_dim, c->layout, &smem);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return PA_ERR_CUDA;
    if (p.tc) {
        // kTcUnitNs, some times what a unit takes, for each unit of a CTA's longest range
        const int64_t tile_units = (int64_t)a.max_blocks * a.B / a.kt + 1 + a.extra;  // max_tiles times this is below 2^31
        const int64_t range = (int64_t)a.Hk * (a.max_tiles * tile_units) / a.C + 1;
        a.wait_ns = kWaitLimitNs + kTcUnitNs * (unsigned long long)std::min(range, (int64_t)1 << 40);
        CUtensorMap tmq, tmk, tmv;
        int32_t gran = gcd(c->block_size, kTcKeys);
        if (!encode_tc_maps(&tmq, &tmk, &tmv, a, c, gran)) return PA_ERR_CUDA;
        void *targs[] = {&tmq, &tmk, &tmv, &a, &gran};
        if (launch_pdl(fn, dim3(p.C), dim3(p.threads), targs, smem, s) != cudaSuccess) return PA_ERR_CUDA;
    } else if (launch_pdl(fn, dim3(p.C), dim3(p.threads), args, smem, s) != cudaSuccess) {
        return PA_ERR_CUDA;
    }
    if ((st = prefill_launch_merge(a, c->dtype == PA_F32, c->head_dim, s)) != PA_OK) return st;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// The call's plan; fits: its scale and alignment suit the tcgen05 kernel.
static pa_status_t prefill_plan_of(const pa_cache_desc_t *c, int32_t N, int32_t T, int32_t H,
                                   const pa_prefill_opts_t *opts, bool fits, PrefillPlan *p) {
    const pa_status_t st = validate_cache_desc(c);
    if (st != PA_OK) return st;
    if (N < 0 || T < 0 || H <= 0 || H % c->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int want = opts ? opts->kernel : PA_KERNEL_AUTO;
    if (want != PA_KERNEL_AUTO && want != PA_KERNEL_SIMT && want != PA_KERNEL_MMA) return PA_ERR_INVALID_ARG;
    if (opts && opts->num_splits < 0) return PA_ERR_INVALID_ARG;
    const int32_t G = H / c->num_kv_heads;
    if (G > 64) return PA_ERR_UNSUPPORTED;
    const bool tc = want != PA_KERNEL_SIMT && fits && tc_supported(c, G);
    if (want == PA_KERNEL_MMA && !tc) return PA_ERR_UNSUPPORTED;
    return prefill_layout(tc, c, N, T, H, opts ? opts->num_splits : 0, p);
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_prefill_workspace_bytes(const pa_cache_desc_t *cache, int32_t num_seqs, int32_t num_tokens,
                                             int32_t num_heads, const pa_prefill_opts_t *opts) try {
    PrefillPlan p;
    if (prefill_plan_of(cache, num_seqs, num_tokens, num_heads, opts, true, &p) != PA_OK) return 0;
    const size_t need = p.total;
    if (!p.tc || (opts && opts->kernel == PA_KERNEL_MMA)) return need;
    // a call whose scale or alignment keeps it from the tcgen05 kernel needs the other layout
    if (prefill_plan_of(cache, num_seqs, num_tokens, num_heads, opts, false, &p) != PA_OK) return 0;
    return std::max(need, p.total);
} catch (...) {
    return 0;
}

extern "C" pa_status_t pa_prefill(void *out, const void *q, const void *k_cache, const void *v_cache,
                                  const pa_cache_desc_t *cache, const int32_t *block_tables,
                                  int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *cu_q_lens,
                                  int32_t num_seqs, int32_t num_tokens, int32_t num_heads, float scale,
                                  void *workspace, size_t workspace_bytes, const pa_prefill_opts_t *opts,
                                  pa_stream_t stream) try {
    PrefillPlan p;
    const bool fits = scale > 0.f && scale < INFINITY && ((uintptr_t)q | (uintptr_t)out) % 16 == 0;
    const pa_status_t st = prefill_plan_of(cache, num_seqs, num_tokens, num_heads, opts, fits, &p);
    if (st != PA_OK) return st;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_q_lens || !workspace)
        return PA_ERR_INVALID_ARG;
    if (max_blocks_per_seq <= 0 || (int64_t)num_seqs * max_blocks_per_seq >= ((int64_t)1 << 31) ||
        (int64_t)max_blocks_per_seq * cache->block_size >= ((int64_t)1 << 31))
        return PA_ERR_INVALID_ARG;
    // the units of a KV head are counted in 32 bits
    if ((int64_t)p.max_tiles * ((int64_t)max_blocks_per_seq * cache->block_size / p.kt + 1 + p.extra) >= ((int64_t)1 << 31))
        return PA_ERR_UNSUPPORTED;
    if (!(scale == scale)) return PA_ERR_INVALID_ARG;
    if (((uintptr_t)workspace & 255) != 0) return PA_ERR_INVALID_ARG;
    if (workspace_bytes < p.total) return PA_ERR_WORKSPACE;
    const int eb = dtype_bytes(cache->dtype);
    if (((uintptr_t)q | (uintptr_t)out) % (size_t)(eb * 2) != 0) return PA_ERR_INVALID_ARG;
    if (((uintptr_t)k_cache | (uintptr_t)v_cache) % 16 != 0) return PA_ERR_INVALID_ARG;
    PrefillArgs a{};
    a.q = q;
    a.out = out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.tables = block_tables;
    a.seq_lens = seq_lens;
    a.cu_q = cu_q_lens;
    a.max_blocks = max_blocks_per_seq;
    a.N = num_seqs;
    a.T = num_tokens;
    a.H = num_heads;
    a.scale_log2 = scale * 1.4426950408889634f;
    return prefill_launch(p, cache, a, workspace, (cudaStream_t)stream);
} catch (...) {
    return host_failure();
}
