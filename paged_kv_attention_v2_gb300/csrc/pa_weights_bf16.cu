// pa_weights_bf16.cu -- kernel instantiations of pa_add_weights for bf16 queries.
#include "pa_weights.cuh"

namespace pa {
bool launch_weights_bf16(WeightParams& p, int head_size, int kv, int sms, void* stream) {
    switch (kv) {
    case kWSame: return launch_weights<__nv_bfloat16, kWSame>(p, head_size, sms, stream);
    case kWE4M3: return launch_weights<__nv_bfloat16, kWE4M3>(p, head_size, sms, stream);
    case kWE5M2: return launch_weights<__nv_bfloat16, kWE5M2>(p, head_size, sms, stream);
    default: return launch_weights<__nv_bfloat16, kWE2M1>(p, head_size, sms, stream);
    }
}
}  // namespace pa
