// pck_paged_token_e4m3_128.cu -- one-token attention over a quantised paged cache: the kernels of D = 128.
#include "pck_paged_token_e4m3_impl.cuh"

namespace pck {

cudaError_t launch_paged_token_e4m3_128(PagedAttn& p, cudaStream_t st) { return launch8_d<128>(p, st); }

}  // namespace pck
