// pck_paged.cu -- head norms with the rotary rotation, and the append to a 16-bit paged cache.
#include "pck_paged_rope_impl.cuh"

namespace pck {

cudaError_t launch_norm_rope(const RopeParams& p, int in_dtype, int cache_dtype, int sms, cudaStream_t st) {
    if (in_dtype == PCK_DT_F16) return launch_t<__half, __half>(p, sms, st);
    if (in_dtype == PCK_DT_BF16) return launch_t<__nv_bfloat16, __nv_bfloat16>(p, sms, st);
    if (cache_dtype == PCK_DT_F16) return launch_t<float, __half>(p, sms, st);
    return launch_t<float, __nv_bfloat16>(p, sms, st);
}

}  // namespace pck
