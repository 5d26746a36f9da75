// Instantiations of the tcgen05 chunk-attention kernel.
#include "prefill_kernels.h"
#include "prefill_tc.cuh"

namespace pa {

template <int D, int kConv>
static const void *tc_for(size_t *smem, int *threads) {
    *smem = TcPrefill<D, kConv>::kSmem;
    *threads = TcPrefill<D, kConv>::kThreads;
    return (const void *)prefill_tc_kernel<D, kConv>;
}
template <int D>
static const void *tc_for(int conv, size_t *smem, int *threads) {
    return conv == 0 ? tc_for<D, 0>(smem, threads) : conv == 4 ? tc_for<D, 4>(smem, threads) : tc_for<D, 8>(smem, threads);
}

const void *prefill_tc_ptr(int D, int conv, size_t *smem, int *threads) {
    return D == 64 ? tc_for<64>(conv, smem, threads) : tc_for<128>(conv, smem, threads);
}

}  // namespace pa
