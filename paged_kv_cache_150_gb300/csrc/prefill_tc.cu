// Instantiations of the tcgen05 chunk-attention kernel.
#include "prefill_kernels.h"
#include "prefill_tc.cuh"

namespace pa {

template <int D, bool kFp8>
static const void *tc_for(size_t *smem, int *threads) {
    *smem = TcPrefill<D, kFp8>::kSmem;
    *threads = TcPrefill<D, kFp8>::kThreads;
    return (const void *)prefill_tc_kernel<D, kFp8>;
}

const void *prefill_tc_ptr(int D, bool fp8, size_t *smem, int *threads) {
    if (D == 64) return fp8 ? tc_for<64, true>(smem, threads) : tc_for<64, false>(smem, threads);
    return fp8 ? tc_for<128, true>(smem, threads) : tc_for<128, false>(smem, threads);
}

}  // namespace pa
