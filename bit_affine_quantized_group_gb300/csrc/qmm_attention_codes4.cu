// Attention over a cache of 4-bit codes.
#include "qmm_attention_codes.cuh"

namespace qmmk {

cudaError_t configure_attention_codes4() { return configure_codes<4>(); }

cudaError_t launch_attention_codes4(int head_dim, const AttnParams& p, int num_sms, cudaStream_t stream) {
    return launch_codes<4>(head_dim, p, num_sms, stream);
}

}  // namespace qmmk
