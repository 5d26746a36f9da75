// Single-query attention over the 8-bit cache (pa_decode_fp8).
#include "fp8_codec.cuh"
#include "prefill_kernels.h"

namespace pa {

static pa_status_t decode_fp8_plan(const pa_cache_desc_t *c, int32_t N, int32_t H, const pa_prefill_opts_t *opts,
                                   PrefillPlan *p) {
    const pa_status_t st = validate_fp8_desc(c);
    if (st != PA_OK) return st;
    if (N < 0 || H <= 0 || H % c->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int want = opts ? opts->kernel : PA_KERNEL_AUTO;
    if (want != PA_KERNEL_AUTO && want != PA_KERNEL_SIMT && want != PA_KERNEL_MMA) return PA_ERR_INVALID_ARG;
    if (opts && opts->num_splits < 0) return PA_ERR_INVALID_ARG;
    if (H / c->num_kv_heads > 8) return PA_ERR_UNSUPPORTED;
    if (want == PA_KERNEL_MMA) return PA_ERR_UNSUPPORTED;
    return prefill_layout(false, c, N, N, H, opts ? opts->num_splits : 0, p);
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_fp8_workspace_bytes(const pa_cache_desc_t *cache, int32_t num_seqs, int32_t num_heads,
                                                const pa_prefill_opts_t *opts) try {
    PrefillPlan p;
    if (decode_fp8_plan(cache, num_seqs, num_heads, opts, &p) != PA_OK) return 0;
    return p.total;
} catch (...) {
    return 0;
}

extern "C" pa_status_t pa_decode_fp8(void *out, const void *q, const void *k_cache, const void *v_cache,
                                     const uint8_t *k_scale, const uint8_t *v_scale, const pa_cache_desc_t *cache,
                                     const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
                                     int32_t num_seqs, int32_t num_heads, float scale, void *workspace,
                                     size_t workspace_bytes, const pa_prefill_opts_t *opts, pa_stream_t stream) try {
    PrefillPlan p;
    const pa_status_t st = decode_fp8_plan(cache, num_seqs, num_heads, opts, &p);
    if (st != PA_OK) return st;
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !seq_lens || !workspace)
        return PA_ERR_INVALID_ARG;
    if (max_blocks_per_seq <= 0 || (int64_t)num_seqs * max_blocks_per_seq >= ((int64_t)1 << 31) ||
        (int64_t)max_blocks_per_seq * cache->block_size >= ((int64_t)1 << 31))
        return PA_ERR_INVALID_ARG;
    if ((int64_t)num_seqs * ((int64_t)max_blocks_per_seq * cache->block_size / p.kt + 1 + p.extra) >= ((int64_t)1 << 31))
        return PA_ERR_UNSUPPORTED;
    if (!(scale == scale)) return PA_ERR_INVALID_ARG;
    if (((uintptr_t)workspace & 255) != 0) return PA_ERR_INVALID_ARG;
    if (workspace_bytes < p.total) return PA_ERR_WORKSPACE;
    if (((uintptr_t)q | (uintptr_t)out) % 4 != 0) return PA_ERR_INVALID_ARG;
    if (((uintptr_t)k_cache | (uintptr_t)v_cache) % 16 != 0) return PA_ERR_INVALID_ARG;
    PrefillArgs a{};
    a.q = q;
    a.out = out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.tables = block_tables;
    a.seq_lens = seq_lens;
    a.max_blocks = max_blocks_per_seq;
    a.N = num_seqs;
    a.T = num_seqs;
    a.H = num_heads;
    a.scale_log2 = scale * 1.4426950408889634f;
    return prefill_launch(p, cache, a, workspace, (cudaStream_t)stream);
} catch (...) {
    return host_failure();
}
