// Parameters and launch of the sampling kernel (sample.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace w4a16 {

constexpr int kSampleMaxVocab = 262144;

struct SampleParams {
    const void* logits;          // [batch][stride], vocab valid
    long long stride;            // elements between rows
    const float* u;              // [batch], in [0, 1)
    const float* temperature;    // [batch] or null: 1
    const int32_t* top_k;        // [batch] or null: none
    const float* top_p;          // [batch] or null: 1
    const float* min_p;          // [batch] or null: 0
    int32_t* token;              // [batch]
    float* prob;                 // [batch] or null
    int batch, vocab;
    int dtype;                   // w4a16_dtype
    int slice;                   // elements of a CTA's slice (set by the launch)
    int in_turn;                 // rows are taken in order of their work, not of their index (set by the launch)
};
cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t stream);

}  // namespace w4a16
