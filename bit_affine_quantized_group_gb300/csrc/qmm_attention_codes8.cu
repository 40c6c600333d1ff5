// Attention over a cache of 8-bit codes.
#include "qmm_attention_codes.cuh"

namespace qmmk {

cudaError_t configure_attention_codes8() { return configure_codes<8>(); }

cudaError_t launch_attention_codes8(int head_dim, const AttnParams& p, int num_sms, cudaStream_t stream) {
    return launch_codes<8>(head_dim, p, num_sms, stream);
}

}  // namespace qmmk
