// Single-query attention over the 8-bit cache (pa_decode_fp8): host side.  The
// tensor-core kernel is decode_fp8.cuh; head_dim 256 and the block sizes it
// does not take run on the CUDA-core kernel of chunk attention with one new
// token per sequence.
#include "decode_fp8.cuh"
#include "prefill_kernels.h"

namespace pa {

namespace {

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// The tensor-core kernel's shape for this cache; false if it does not take it.
bool f8_shape(const pa_cache_desc_t *c, int G, F8Args *f, size_t *smem) {
    const int D = c->head_dim, Hk = c->num_kv_heads;
    if ((D != 64 && D != 128) || c->block_size % 8 != 0 || Hk > 256) return false;
    f->Hk = Hk;
    f->G = G;
    f->NH = Hk % 8 == 0 ? 8 : Hk % 4 == 0 ? 4 : Hk % 2 == 0 ? 2 : 1;
    f->T = kF8Warps * 16 / f->NH;
    f->gran = gcd(c->block_size, f->T);
    if (f->gran * Hk % 16 != 0) return false;  // a box's scale bytes are copied in 16-byte pieces
    f->scale_bytes = (uint32_t)(f->T * Hk);
    auto bytes = [&](int stages) {
        return D == 128 ? F8Smem<128>::bytes(stages, f->scale_bytes, f->NH, G)
                        : F8Smem<64>::bytes(stages, f->scale_bytes, f->NH, G);
    };
    // 64 KiB of codes in flight per CTA, 128 per SM (96 and 192 were 2% slower)
    f->stages = D == 128 ? 2 : 4;
    *smem = bytes(f->stages);
    return *smem <= 112 * 1024;
}

const void *f8_kernel(int D) {
    return D == 128 ? (const void *)decode_fp8_kernel<128> : (const void *)decode_fp8_kernel<64>;
}

struct F8Plan {
    PrefillPlan p;
    F8Args f;
    bool mma;
};

pa_status_t decode_fp8_plan(const pa_cache_desc_t *c, int32_t N, int32_t H, const pa_prefill_opts_t *opts, bool aligned,
                            F8Plan *pl) {
    const pa_status_t st = validate_fp8_desc(c);
    if (st != PA_OK) return st;
    if (N < 0 || H <= 0 || H % c->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int want = opts ? opts->kernel : PA_KERNEL_AUTO;
    if (want != PA_KERNEL_AUTO && want != PA_KERNEL_SIMT && want != PA_KERNEL_MMA) return PA_ERR_INVALID_ARG;
    if (opts && opts->num_splits < 0) return PA_ERR_INVALID_ARG;
    const int G = H / c->num_kv_heads;
    if (G > 8) return PA_ERR_UNSUPPORTED;
    const int32_t splits = opts ? opts->num_splits : 0;
    size_t smem = 0;
    pl->mma = want != PA_KERNEL_SIMT && aligned && f8_shape(c, G, &pl->f, &smem);
    if (!pl->mma) return want == PA_KERNEL_MMA ? PA_ERR_UNSUPPORTED : prefill_layout(false, c, N, N, H, splits, &pl->p);
    PrefillPlan &p = pl->p;
    p.tc = false;
    p.rows = kF8SlotRows;
    p.nrt = 1;
    p.tq1 = 1;
    p.kt = pl->f.T;
    p.extra = kF8Extra;
    p.threads = kF8Threads;
    p.max_tiles = N;
    p.smem = smem;
    p.C = splits > 0 ? splits : default_ctas(f8_kernel(c->head_dim), kF8Threads, smem);
    if (p.C <= 0) return PA_ERR_CUDA;
    prefill_workspace(&p, N, c->head_dim);
    return PA_OK;
}

// {D codes, NB * B rows, Hk heads} in boxes of gran rows x NH heads.
bool encode_codes_map(CUtensorMap *m, const void *base, const pa_cache_desc_t *c, const F8Args &f) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t D = c->head_dim;
    const cuuint64_t dims[3] = {D, (cuuint64_t)c->num_blocks * c->block_size, (cuuint64_t)c->num_kv_heads};
    const cuuint64_t strides[2] = {(cuuint64_t)c->num_kv_heads * D, D};
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)f.gran, (cuuint32_t)f.NH}, one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_fp8_workspace_bytes(const pa_cache_desc_t *cache, int32_t num_seqs, int32_t num_heads,
                                                const pa_prefill_opts_t *opts) try {
    F8Plan pl;
    if (decode_fp8_plan(cache, num_seqs, num_heads, opts, true, &pl) != PA_OK) return 0;
    const size_t need = pl.p.total;
    if (!pl.mma || (opts && opts->kernel == PA_KERNEL_MMA)) return need;
    // a call whose scale bytes are not aligned needs the CUDA-core layout
    if (decode_fp8_plan(cache, num_seqs, num_heads, opts, false, &pl) != PA_OK) return 0;
    return std::max(need, pl.p.total);
} catch (...) {
    return 0;
}

extern "C" pa_status_t pa_decode_fp8(void *out, const void *q, const void *k_cache, const void *v_cache,
                                     const uint8_t *k_scale, const uint8_t *v_scale, const pa_cache_desc_t *cache,
                                     const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
                                     int32_t num_seqs, int32_t num_heads, float scale, void *workspace,
                                     size_t workspace_bytes, const pa_prefill_opts_t *opts, pa_stream_t stream) try {
    F8Plan pl;
    const bool aligned = ((uintptr_t)k_scale | (uintptr_t)v_scale) % 16 == 0;
    pa_status_t st = decode_fp8_plan(cache, num_seqs, num_heads, opts, aligned, &pl);
    if (st != PA_OK) return st;
    const PrefillPlan &p = pl.p;
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
    cudaStream_t s = (cudaStream_t)stream;
    if (!pl.mma) return prefill_launch(p, cache, a, workspace, s);
    const F8Args &f = pl.f;
    a.Hk = f.Hk / f.NH;  // the list's outer index: head groups
    a.G = f.NH * f.G;
    a.NB = cache->num_blocks;
    a.B = cache->block_size;
    if ((st = prefill_bind(p, &a, workspace)) != PA_OK) return st;
    CUtensorMap tmk, tmv;
    if (!encode_codes_map(&tmk, k_cache, cache, f) || !encode_codes_map(&tmv, v_cache, cache, f)) return PA_ERR_CUDA;
    const void *fn = f8_kernel(cache->head_dim);
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem) != cudaSuccess)
        return PA_ERR_CUDA;
    cudaGetLastError();
    if ((st = prefill_launch_plan(a, s)) != PA_OK) return st;
    F8Args fv = f;
    void *args[] = {&tmk, &tmv, &a, &fv};
    if (launch_pdl(fn, dim3(p.C), dim3(kF8Threads), args, p.smem, s) != cudaSuccess) return PA_ERR_CUDA;
    if ((st = prefill_launch_merge(a, false, cache->head_dim, s)) != PA_OK) return st;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
} catch (...) {
    return host_failure();
}
