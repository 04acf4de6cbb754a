// serve_internal.cuh -- launchers of the operators of a decoding step (the layer for a few tokens, the
// choice of the next token), shared by their kernels and the C ABI. Not part of the public C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "moe_internal.cuh"

namespace moe {

// The layer for a few tokens (few_tokens.cu): tokens are the columns of its products, up to four tiles of
// eight, and the bits of a 32-bit mask per expert; a (token, expert) pair's score and H row are looked up in
// shared memory.
constexpr int kFewMaxTokens = 32;
constexpr int kFewMaxPairs = 512;

struct FewProblem {
    const void* x;        // bf16 [T, D]
    const int32_t* ids;   // [T, K], or null: chosen from the logits
    const void* scores;   // [T, K] fp32 or bf16
    int32_t scores_dtype;
    const void* logits;   // [T, E] fp32 or bf16
    int32_t logits_dtype;
    bool normalize;
    int32_t* ids_out;     // [T, K], with logits
    float* scores_out;    // [T, K]
    const void* w13;      // bf16 [E, 2, F, D]
    const void* w2;       // bf16 [E, D, F]
    void* out;            // bf16 [T, D]
    uint32_t* status;
    void* h;              // bf16 [2, T*K, F]: H in two parts
    int32_t T, D, F, E, K;
    int sm_count;
};
moe_status_t launch_few(const FewProblem& p, cudaStream_t stream);

// The choice of the next token (sample.cu).
constexpr int32_t kSampleMaxV = 1 << 24;
struct SampleProblem {
    const void* logits;        // [T, V] of dtype
    int32_t dtype;
    const float* uniform;      // [T]
    const float* temperature;  // [T] each, or null
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* token;            // [T]
    float* logprob;            // [T] or null
    int64_t T;
    int32_t V;
    int sm_count;
};
moe_status_t launch_sample(const SampleProblem& p, cudaStream_t stream);

}  // namespace moe
