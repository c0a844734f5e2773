// pa_family_f16_fp4.cu -- kernel instantiations for an fp16 query with a 4-bit (E2M1) KV cache.
#include "pa_launch.cuh"

namespace pa {
cudaError_t launch_f16_fp4(const Params& p, const LaunchArgs& la) { return launch_family_fp4<__half>(p, la); }
}  // namespace pa
