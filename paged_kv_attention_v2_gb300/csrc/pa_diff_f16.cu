// pa_diff_f16.cu -- kernel instantiations of differential attention for f16
// inputs and caches.
#include "pa_launch.cuh"

namespace pa {
cudaError_t launch_diff_f16(const Params& p, const LaunchArgs& la) {
    return la.head_size == 256 ? launch_diff_family<__half, kKvSame, 256>(p, la)
                               : launch_diff_family<__half, kKvSame, 128>(p, la);
}
}  // namespace pa
