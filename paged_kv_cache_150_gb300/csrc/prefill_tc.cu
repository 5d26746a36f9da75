// Instantiations of the tcgen05 chunk-attention kernel.
#include "prefill_kernels.h"
#include "prefill_tc.cuh"

namespace pa {

const void *prefill_tc_ptr(int D, size_t *smem) {
    if (D == 64) {
        *smem = TcPrefill<64>::kSmem;
        return (const void *)prefill_tc_kernel<64>;
    }
    *smem = TcPrefill<128>::kSmem;
    return (const void *)prefill_tc_kernel<128>;
}

}  // namespace pa
