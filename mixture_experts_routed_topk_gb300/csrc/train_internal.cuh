// train_internal.cuh -- launchers of the operators around the expert layer (layer norm, top-k
// router, vocabulary losses), shared by their kernels and the C ABI. Not part of the public C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "moe_internal.cuh"

namespace moe {

// Element types of the layer norm and router entry points (MOE_DTYPE_*).
inline size_t dtype_size(int32_t d) { return d == MOE_DTYPE_F32 ? 4 : 2; }

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct LayerNormProblem {
    const void* x;
    const void* gamma;  // may be null: 1
    const void* beta;   // may be null: 0 (forward)
    int32_t dtype, param_dtype;
    void* y;
    float* mean;
    float* rstd;
    // backward
    const void* dy;
    const float* mean_in;
    const float* rstd_in;
    void* dx;
    void* dgamma;    // may be null
    void* dbeta;     // may be null
    float* partial;  // [kLnMaxBlocks][2][D] fp32
    int64_t T;
    int32_t D;
    float eps;
    int sm_count;
};
// Rows of the parameter-gradient partials: the backward grid has at most this many blocks, which
// the workspace size is computed from without asking the device.
constexpr int kLnMaxBlocks = 152;
constexpr int32_t kLnMaxD = 1 << 24;

moe_status_t launch_layernorm_fwd(const LayerNormProblem& p, cudaStream_t stream);
moe_status_t launch_layernorm_bwd(const LayerNormProblem& p, cudaStream_t stream);

struct RouterProblem {
    const void* logits;  // [T, E] fp32 or bf16
    int32_t dtype;
    int64_t T;
    int32_t E, K;
    bool normalize;
    int32_t* ids;
    float* scores;
    const int32_t* ids_in;
    const float* dscores;
    void* dlogits;
};
moe_status_t launch_router_fwd(const RouterProblem& p, cudaStream_t stream);
moe_status_t launch_router_bwd(const RouterProblem& p, cudaStream_t stream);

// Vocabulary losses of a linear head (lm_loss.cu).
struct LmProblem {
    const void* x;  // bf16 [T, D]
    const void* w;  // bf16 [V, D]
    int64_t T;
    int32_t D, V, K;
    const int32_t* targets;  // cross entropy: [T] (teacher_ids null)
    int32_t ignore_index;
    const int32_t* teacher_ids;   // distillation: [T, K]
    const float* teacher_logits;  // [T, K]
    float temperature;
    float* loss;
    float* lse;
    const float* lse_in;
    const float* dloss;
    void* dx;  // may be null
    void* dw;  // may be null
    uint8_t* ws;
    int sm_count;
};
// Workspace bytes, or 0 for sizes outside the limits.
size_t lm_workspace_bytes(int64_t T, int32_t D, int32_t V, int32_t K);
moe_status_t launch_lm_fwd(const LmProblem& p, cudaStream_t stream);
moe_status_t launch_lm_bwd(const LmProblem& p, cudaStream_t stream);

}  // namespace moe
