// pck_paged_token_e4m3_wide.cu -- one-token attention over a quantised paged cache: the kernels of D = 192, 256.
#include "pck_paged_token_e4m3_impl.cuh"

namespace pck {

cudaError_t launch_paged_token_e4m3_wide(PagedAttn& p, int D, cudaStream_t st) {
    return D == 192 ? launch8_d<192>(p, st) : D == 256 ? launch8_d<256>(p, st) : cudaErrorInvalidValue;
}

}  // namespace pck
