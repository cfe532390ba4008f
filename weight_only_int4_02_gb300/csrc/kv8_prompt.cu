// The tcgen05 attention kernel over the 8-bit cache.
#include "kv_prompt.cuh"

namespace w4a16 {

size_t kv8_prompt_partial_bytes(int sms) { return prompt::partial_bytes(sms); }

cudaError_t setup_kv8_prompt() { return prompt::setup<8>(); }

cudaError_t launch_kv8_prompt(const Kv4AttnParams& p, int head_dim, int sms, cudaStream_t stream)
{
    return prompt::launch<8>(p, head_dim, sms, stream);
}

}  // namespace w4a16
