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

// The float's position in the order of the reals as an unsigned integer; never 0. The addition makes
// -0 equal to +0 and every NaN the canonical one, whose key is the largest.
__device__ __forceinline__ uint32_t order_key(float v) {
    const int32_t b = __float_as_int(v + 0.0f);
    return static_cast<uint32_t>(b ^ ((b >> 31) | INT32_MIN));
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
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

// The norms before and after a block with its gate and residual scale (block_norm_*.cu).
struct BlockNormProblem {
    const void* block;       // [T, D]; backward: may be null where its gradient does not need it
    const void* residual;    // forward
    const void* post_gamma;  // [D] or null: 1
    const void* gate;        // [D] of param_dtype, [T, D] of dtype, or null: 1
    const void* pre_gamma;   // [D] or null: 1
    bool gate_per_token;
    int32_t dtype, param_dtype;
    void* stream;    // forward: written; backward: read
    void* normed;
    float* post_rstd;  // null: no norm after the block
    float* pre_rstd;
    // backward
    const void* dstream;  // may be null: 0
    const void* dnormed;
    const float* post_rstd_in;
    const float* pre_rstd_in;
    void* dblock;
    void* dresidual;
    void* dpost_gamma;  // these may be null
    void* dgate;
    void* dpre_gamma;
    float* partial;  // [kBnMaxBlocks][2][D] fp32
    int64_t T;
    int32_t D;
    float residual_scale, eps;
    int sm_count;
};
// Rows of the parameter gradients' partial sums, as for the layer norm; long rows have two blocks to an SM.
constexpr int kBnMaxBlocks = 304;

moe_status_t launch_block_norm_fwd(const BlockNormProblem& p, cudaStream_t stream);
moe_status_t launch_block_norm_bwd(const BlockNormProblem& p, cudaStream_t stream);

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
