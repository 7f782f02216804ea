// logprobs.cuh -- argument block and launcher of the token log probabilities
// (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mtp {

struct LogprobArgs {
    const void* logits;
    long long rows, V, stride;
    const int32_t* tokens;
    int K;
    float *logprob, *entropy;
    int32_t* top_ids;
    float* top_logprobs;
    unsigned long long timeout_ns;   // of a wait inside the kernel
};
cudaError_t launch_logprobs(const LogprobArgs& a, int ldtype, int sms, cudaStream_t s);

}  // namespace mtp
