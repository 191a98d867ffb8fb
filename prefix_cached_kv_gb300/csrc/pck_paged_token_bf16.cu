// pck_paged_token_bf16.cu -- one-token attention over a paged cache: the bf16 kernels.
#include "pck_paged_token_impl.cuh"

namespace pck {

cudaError_t launch_paged_token_bf16(PagedAttn& p, int D, cudaStream_t st) { return launch_d<__nv_bfloat16>(p, D, st); }

}  // namespace pck
