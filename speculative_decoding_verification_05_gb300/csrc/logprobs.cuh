// Parameters of the log-probability kernel (logprobs.cu).
#pragma once

#include "common.cuh"

namespace sv {

struct LogprobParams {
    const void* logits;     // [B, P, V]
    const int32_t* tokens;  // [B, P]; -1: no token, the row is not read
    long long rows;         // B * P
    int P, V, top;
    float c2, inv_t;        // log2(e) / T, 1 / T
    float* logprob;         // [B, P]
    int32_t* rank;          // [B, P] or null
    float* entropy;         // [B, P] or null
    int32_t* top_tokens;    // [B, P, top]
    float* top_logprobs;    // [B, P, top]
    int32_t* status;        // [B] or null; zero at the launch where P > 1
    int parts, part_granules;  // CTAs of a row, 16-byte granules of each (set by the launcher)
};

cudaError_t launch_logprobs(const LogprobParams& p, int dtype, cudaStream_t st);
cudaError_t debug_read_logprobs(unsigned int* count, unsigned int* line);

}  // namespace sv
