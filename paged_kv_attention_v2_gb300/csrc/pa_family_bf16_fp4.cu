// pa_family_bf16_fp4.cu -- kernel instantiations for a bf16 query with a 4-bit (E2M1) KV cache.
#include "pa_launch.cuh"

namespace pa {
cudaError_t launch_bf16_fp4(const Params& p, const LaunchArgs& la) { return launch_family_fp4<__nv_bfloat16>(p, la); }
}  // namespace pa
