// Host handles of the chunk-attention kernels (instantiated in prefill_simt.cu
// and prefill_tc.cu) and the call that launches the CUDA-core one, shared by
// pa_prefill and pa_decode_fp8.
#pragma once

#include "prefill_plan.cuh"

namespace pa {

// Shape of one call: which kernel, its tiles, and the workspace behind it.
struct PrefillPlan {
    bool tc;           // tcgen05 kernel
    int32_t rows, nrt; // query rows of a row tile, row tiles per tile
    int32_t tq1;       // tokens per row tile
    int32_t kt;        // keys per unit
    int32_t extra;     // weight of a tile beside its units
    int32_t threads;   // of an attention CTA
    int32_t C, max_tiles;
    size_t smem;
    size_t off_ctl, off_tile0, off_cu, off_tiles, off_start, off_merges, off_ml, off_acc, total;
};

// Kernel and shared memory of prefill_simt_kernel for a cache element type
// (q and out: fp32 for PA_F32, else bf16), head_dim and layout; nullptr if none.
const void *prefill_simt_ptr(int cache_dtype, int D, int layout, size_t *smem);

// prefill_tc_kernel for head_dim 64 or 128.
const void *prefill_tc_ptr(int D, size_t *smem);

// Lays out a call of the CUDA-core kernel (tc false) or the tcgen05 one.
pa_status_t prefill_layout(bool tc, const pa_cache_desc_t *c, int32_t N, int32_t T, int32_t H, int32_t num_splits,
                           PrefillPlan *p);

// The workspace behind p's shape (tiles, units, CTAs set) and head_dim.
void prefill_workspace(PrefillPlan *p, int32_t N, int32_t head_dim);

// Fills in the plan's part of a call's arguments; PA_ERR_CUDA without an error word.
pa_status_t prefill_bind(const PrefillPlan &p, PrefillArgs *a, void *workspace);

// Enqueue the work list, and the merge of the pieces (fp32 or bf16 output).
pa_status_t prefill_launch_plan(PrefillArgs &a, cudaStream_t s);
pa_status_t prefill_launch_merge(PrefillArgs &a, bool f32, int32_t head_dim, cudaStream_t s);

// Enqueues the work list, the attention and the merge.  a holds the call's
// arguments; the plan's fields and the workspace pointers are filled in here.
pa_status_t prefill_launch(const PrefillPlan &p, const pa_cache_desc_t *c, PrefillArgs a, void *workspace,
                           cudaStream_t s);

}  // namespace pa
