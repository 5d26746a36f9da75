// Instantiations of the tcgen05 chunk-attention kernel.
#include "prefill_kernels.h"
#include "prefill_tc.cuh"

namespace pa {

template <int D, int kConv, bool kPair>
static const void *tc_for(size_t *smem, int *threads) {
    *smem = TcPrefill<D, kConv, kPair>::kSmem;
    *threads = TcPrefill<D, kConv, kPair>::kThreads;
    return (const void *)prefill_tc_kernel<D, kConv, kPair>;
}
template <int D>
static const void *tc_for(int conv, bool pair, size_t *smem, int *threads) {
    return conv == 8   ? tc_for<D, 8, true>(smem, threads)
           : conv == 4 ? tc_for<D, 4, false>(smem, threads)
           : pair      ? tc_for<D, 0, true>(smem, threads)
                       : tc_for<D, 0, false>(smem, threads);
}

const void *prefill_tc_ptr(int D, int conv, bool pair, size_t *smem, int *threads) {
    return D == 64 ? tc_for<64>(conv, pair, smem, threads) : tc_for<128>(conv, pair, smem, threads);
}

}  // namespace pa
