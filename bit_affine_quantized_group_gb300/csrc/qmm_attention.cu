// Attention over a cache of bfloat16, and the choice among the kinds of caches.
#include "qmm_attention.cuh"

namespace qmmk {

cudaError_t configure_attention() {
    cudaError_t e = configure_bits<16>();
    if (e == cudaSuccess) e = configure_attention_codes8();
    if (e == cudaSuccess) e = configure_attention_codes4();
    return e;
}

cudaError_t launch_attention(int head_dim, int bits, const AttnParams& p, int num_sms, cudaStream_t stream) {
    if (bits == 8) return launch_attention_codes8(head_dim, p, num_sms, stream);
    if (bits == 4) return launch_attention_codes4(head_dim, p, num_sms, stream);
    return launch_bits<16>(head_dim, p, num_sms, stream);
}

}  // namespace qmmk
