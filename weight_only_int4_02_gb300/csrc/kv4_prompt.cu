// The tcgen05 attention kernel over the 4-bit cache.
#include "kv_prompt.cuh"

namespace w4a16 {

size_t kv4_prompt_partial_bytes(int sms) { return prompt::partial_bytes(sms); }

cudaError_t setup_kv4_prompt() { return prompt::setup<4>(); }

cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, int head_dim, int sms, cudaStream_t stream)
{
    return prompt::launch<4>(p, head_dim, sms, stream);
}

}  // namespace w4a16
