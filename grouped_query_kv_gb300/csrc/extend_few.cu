// extend_few.cu -- the paged prompt attention of prefill.cuh for calls whose
// requests bring few tokens each, in a unit of its own so that the kernels
// compile side by side.
#include "prefill.cuh"

namespace kvattn {

cudaError_t launch_extend_few(int D, const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                              const void *params, int num_ctas, cudaStream_t stream, const CUtensorMap &tmq4) {
    const PagedPrefillParams &p = *static_cast<const PagedPrefillParams *>(params);
    return D == 64 ? launch_pf<64, true, true>(tmq, tmk, tmv, p, num_ctas, stream, tmq4)
                   : launch_pf<128, true, true>(tmq, tmk, tmv, p, num_ctas, stream, tmq4);
}

}  // namespace kvattn
