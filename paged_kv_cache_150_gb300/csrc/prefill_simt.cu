// Instantiations of the CUDA-core chunk-attention kernel.
#include "prefill_kernels.h"
#include "prefill_simt.cuh"

namespace pa {

template <typename T, typename CT, int LAYOUT>
static const void *simt_for(int D, size_t *smem) {
    switch (D) {
        case 64: *smem = SimtSmem<64, simt_pipe<CT, 64, LAYOUT>()>::kBytes; return (const void *)prefill_simt_kernel<T, CT, 64, LAYOUT>;
        case 128: *smem = SimtSmem<128, simt_pipe<CT, 128, LAYOUT>()>::kBytes; return (const void *)prefill_simt_kernel<T, CT, 128, LAYOUT>;
        case 256: *smem = SimtSmem<256, simt_pipe<CT, 256, LAYOUT>()>::kBytes; return (const void *)prefill_simt_kernel<T, CT, 256, LAYOUT>;
    }
    return nullptr;
}

const void *prefill_simt_ptr(int cache_dtype, int D, int layout, size_t *smem) {
    if (cache_dtype == PA_FP8_E4M3) return simt_for<__nv_bfloat16, CacheE4m3, PA_LAYOUT_ROW>(D, smem);
    if (cache_dtype == PA_FP8_E4M3_BLOCK) return simt_for<__nv_bfloat16, CacheE4m3Block, PA_LAYOUT_ROW>(D, smem);
    if (cache_dtype == PA_F32)
        return layout == PA_LAYOUT_ROW ? simt_for<float, float, PA_LAYOUT_ROW>(D, smem)
                                       : simt_for<float, float, PA_LAYOUT_SPLIT>(D, smem);
    return layout == PA_LAYOUT_ROW ? simt_for<__nv_bfloat16, __nv_bfloat16, PA_LAYOUT_ROW>(D, smem)
                                   : simt_for<__nv_bfloat16, __nv_bfloat16, PA_LAYOUT_SPLIT>(D, smem);
}

}  // namespace pa
