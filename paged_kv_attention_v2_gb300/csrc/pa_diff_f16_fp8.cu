// pa_diff_f16_fp8.cu -- kernel instantiations of differential attention for a
// f16 query with an fp8 (E4M3 or E5M2) KV cache.
#include "pa_launch.cuh"

namespace pa {
cudaError_t launch_diff_f16_fp8(const Params& p, const LaunchArgs& la, int kv) {
    if (la.head_size == 256)
        return kv == kKvE4M3 ? launch_diff_family<__half, kKvE4M3, 256>(p, la)
                             : launch_diff_family<__half, kKvE5M2, 256>(p, la);
    return kv == kKvE4M3 ? launch_diff_family<__half, kKvE4M3, 128>(p, la)
                         : launch_diff_family<__half, kKvE5M2, 128>(p, la);
}
}  // namespace pa
