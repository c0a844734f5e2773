// pa_diff_bf16.cu -- kernel instantiations of differential attention for bf16
// inputs and caches.
#include "pa_launch.cuh"

namespace pa {
cudaError_t launch_diff_bf16(const Params& p, const LaunchArgs& la) {
    return la.head_size == 256 ? launch_diff_family<__nv_bfloat16, kKvSame, 256>(p, la)
                               : launch_diff_family<__nv_bfloat16, kKvSame, 128>(p, la);
}
}  // namespace pa
