// train_api.cu -- the C ABI of the operators around the expert layer (layer norm, top-k router,
// vocabulary losses): argument checks, then the launches. As in moe_api.cu, the checks that need no
// GPU run first, and an entry point only enqueues work on the caller's stream.
#include <cuda_runtime.h>

#include "train_internal.cuh"

namespace moe {
namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool bad_dtype(int32_t d) { return d != MOE_DTYPE_F32 && d != MOE_DTYPE_BF16 && d != MOE_DTYPE_F16; }

moe_status_t sm103(DeviceInfo* dev) {
    const moe_status_t st = device_info(dev);
    if (st != MOE_OK) return st;
    return dev->supported ? MOE_OK : MOE_ERR_UNSUPPORTED_DEVICE;
}

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;

// The checks of the four vocabulary-loss calls (T = 0 asks for no pointers).
moe_status_t check_lm(const LmProblem& p, size_t workspace_bytes, bool backward) {
    if (p.T < 0 || p.D <= 0 || p.V <= 0 || p.K <= 0) return MOE_ERR_INVALID_ARG;
    // the loss has the square as a factor and the logits the reciprocal: past this they leave fp32
    if (!(p.temperature >= 0x1p-60f && p.temperature <= 0x1p60f)) return MOE_ERR_INVALID_ARG;
    const size_t need = lm_workspace_bytes(p.T > 0 ? p.T : 1, p.D, p.V, p.K);
    if (need == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(p.dw, 16)) return MOE_ERR_MISALIGNED;
    if (p.T == 0) return MOE_OK;
    if (!p.x || !p.w || !p.ws) return MOE_ERR_INVALID_ARG;
    if (!p.targets && !(p.teacher_ids && p.teacher_logits)) return MOE_ERR_INVALID_ARG;
    if (backward ? (!p.lse_in || !p.dloss) : (!p.loss || !p.lse)) return MOE_ERR_INVALID_ARG;
    if (!aligned(p.x, 16) || !aligned(p.w, 16) || !aligned(p.dx, 16) || !aligned(p.ws, 256) ||
        !aligned(p.targets, 4) || !aligned(p.teacher_ids, 4) || !aligned(p.teacher_logits, 4) || !aligned(p.loss, 4) ||
        !aligned(p.lse, 4) || !aligned(p.lse_in, 4) || !aligned(p.dloss, 4))
        return MOE_ERR_MISALIGNED;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    return MOE_OK;
}

moe_status_t run_lm(LmProblem& p, size_t workspace_bytes, bool backward, moe_stream_t stream) {
    moe_status_t st = check_lm(p, workspace_bytes, backward);
    if (st != MOE_OK) return st;
    // nothing to compute: no rows (but a zero gradient for the weights), or no gradient asked for
    if (p.T == 0 && !(backward && p.dw)) return MOE_OK;
    if (backward && !p.dx && !p.dw) return MOE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    DeviceInfo dev;
    if ((st = sm103(&dev)) != MOE_OK) return st;
    p.sm_count = dev.sm_count;
    if (p.T == 0) return cudaMemsetAsync(p.dw, 0, 2ull * p.V * p.D, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    return backward ? launch_lm_bwd(p, s) : launch_lm_fwd(p, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_layernorm_fwd(const void* x, const void* gamma, const void* beta, int32_t dtype, int32_t param_dtype,
                               void* y, float* mean, float* rstd, int64_t T, int32_t D, float eps,
                               moe_stream_t stream) {
    if (bad_dtype(dtype) || bad_dtype(param_dtype) || !(eps >= 0.0f) || T < 0 || D <= 0) return MOE_ERR_INVALID_ARG;
    if (T > kMaxRows || D > kLnMaxD) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x || !y || !mean || !rstd) return MOE_ERR_INVALID_ARG;
    const size_t a = dtype_size(dtype), pa = dtype_size(param_dtype);
    if (!aligned(x, a) || !aligned(y, a) || !aligned(gamma, pa) || !aligned(beta, pa) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return MOE_ERR_MISALIGNED;
    DeviceInfo dev;
    const moe_status_t st = sm103(&dev);
    if (st != MOE_OK) return st;
    LayerNormProblem p{};
    p.x = x;
    p.gamma = gamma;
    p.beta = beta;
    p.dtype = dtype;
    p.param_dtype = param_dtype;
    p.y = y;
    p.mean = mean;
    p.rstd = rstd;
    p.T = T;
    p.D = D;
    p.eps = eps;
    p.sm_count = dev.sm_count;
    return launch_layernorm_fwd(p, reinterpret_cast<cudaStream_t>(stream));
}

size_t moe_layernorm_bwd_workspace_bytes(int64_t T, int32_t D) {
    if (T <= 0 || T > kMaxRows || D <= 0 || D > kLnMaxD) return 0;
    return sizeof(float) * 2 * static_cast<size_t>(kLnMaxBlocks) * D;
}

moe_status_t moe_layernorm_bwd(const void* dy, const void* x, const void* gamma, const float* mean, const float* rstd,
                               int32_t dtype, int32_t param_dtype, void* dx, void* dgamma, void* dbeta, int64_t T,
                               int32_t D, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    if (bad_dtype(dtype) || bad_dtype(param_dtype) || T < 0 || D <= 0) return MOE_ERR_INVALID_ARG;
    if (T > kMaxRows || D > kLnMaxD) return MOE_ERR_UNSUPPORTED_SHAPE;
    const size_t a = dtype_size(dtype), pa = dtype_size(param_dtype);
    if (!aligned(dgamma, pa) || !aligned(dbeta, pa)) return MOE_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    DeviceInfo dev;
    moe_status_t st;
    if (T == 0) {  // no rows: the parameters' gradients are zero
        if (!dgamma && !dbeta) return MOE_OK;
        if ((st = sm103(&dev)) != MOE_OK) return st;
        if ((dgamma && cudaMemsetAsync(dgamma, 0, pa * D, s) != cudaSuccess) ||
            (dbeta && cudaMemsetAsync(dbeta, 0, pa * D, s) != cudaSuccess))
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!dy || !x || !mean || !rstd || !dx) return MOE_ERR_INVALID_ARG;
    if (!aligned(dy, a) || !aligned(x, a) || !aligned(dx, a) || !aligned(gamma, pa) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return MOE_ERR_MISALIGNED;
    if (dgamma || dbeta) {  // the partial sums of the parameters' gradients
        if (!workspace) return MOE_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
        if (workspace_bytes < moe_layernorm_bwd_workspace_bytes(T, D)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    if ((st = sm103(&dev)) != MOE_OK) return st;
    LayerNormProblem p{};
    p.x = x;
    p.gamma = gamma;
    p.dtype = dtype;
    p.param_dtype = param_dtype;
    p.dy = dy;
    p.mean_in = mean;
    p.rstd_in = rstd;
    p.dx = dx;
    p.dgamma = dgamma;
    p.dbeta = dbeta;
    p.partial = static_cast<float*>(workspace);
    p.T = T;
    p.D = D;
    p.sm_count = dev.sm_count;
    return launch_layernorm_bwd(p, s);
}

moe_status_t moe_router_topk_fwd(const void* logits, int32_t dtype, int32_t* topk_ids, float* topk_scores, int64_t T,
                                 int32_t E, int32_t K, int32_t normalize, moe_stream_t stream) {
    if ((dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) || T < 0 || E <= 0 || K <= 0 || K > E)
        return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || T > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_ids || !topk_scores) return MOE_ERR_INVALID_ARG;
    if (!aligned(logits, dtype_size(dtype)) || !aligned(topk_ids, 4) || !aligned(topk_scores, 4))
        return MOE_ERR_MISALIGNED;
    DeviceInfo dev;
    const moe_status_t st = sm103(&dev);
    if (st != MOE_OK) return st;
    RouterProblem p{};
    p.logits = logits;
    p.dtype = dtype;
    p.T = T;
    p.E = E;
    p.K = K;
    p.normalize = normalize != 0;
    p.ids = topk_ids;
    p.scores = topk_scores;
    return launch_router_fwd(p, reinterpret_cast<cudaStream_t>(stream));
}

moe_status_t moe_router_topk_bwd(const void* logits, int32_t dtype, const int32_t* topk_ids, const float* dscores,
                                 void* dlogits, int64_t T, int32_t E, int32_t K, int32_t normalize,
                                 moe_stream_t stream) {
    if ((dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) || T < 0 || E <= 0 || K <= 0 || K > E)
        return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || T > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_ids || !dscores || !dlogits) return MOE_ERR_INVALID_ARG;
    if (!aligned(logits, dtype_size(dtype)) || !aligned(dlogits, dtype_size(dtype)) || !aligned(topk_ids, 4) ||
        !aligned(dscores, 4))
        return MOE_ERR_MISALIGNED;
    DeviceInfo dev;
    const moe_status_t st = sm103(&dev);
    if (st != MOE_OK) return st;
    RouterProblem p{};
    p.logits = logits;
    p.dtype = dtype;
    p.T = T;
    p.E = E;
    p.K = K;
    p.normalize = normalize != 0;
    p.ids_in = topk_ids;
    p.dscores = dscores;
    p.dlogits = dlogits;
    return launch_router_bwd(p, reinterpret_cast<cudaStream_t>(stream));
}

size_t moe_lm_workspace_bytes(int64_t T, int32_t D, int32_t V, int32_t K) { return lm_workspace_bytes(T, D, V, K); }

moe_status_t moe_lm_ce_fwd(const void* x, const void* w, const int32_t* targets, int32_t ignore_index, float* loss,
                           float* lse, int64_t T, int32_t D, int32_t V, void* workspace, size_t workspace_bytes,
                           moe_stream_t stream) {
    LmProblem p{};
    p.x = x;
    p.w = w;
    p.T = T;
    p.D = D;
    p.V = V;
    p.K = 1;
    p.targets = targets;
    p.ignore_index = ignore_index;
    p.temperature = 1.0f;
    p.loss = loss;
    p.lse = lse;
    p.ws = static_cast<uint8_t*>(workspace);
    return run_lm(p, workspace_bytes, false, stream);
}

moe_status_t moe_lm_ce_bwd(const void* x, const void* w, const int32_t* targets, int32_t ignore_index,
                           const float* lse, const float* dloss, void* dx, void* dw, int64_t T, int32_t D, int32_t V,
                           void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    LmProblem p{};
    p.x = x;
    p.w = w;
    p.T = T;
    p.D = D;
    p.V = V;
    p.K = 1;
    p.targets = targets;
    p.ignore_index = ignore_index;
    p.temperature = 1.0f;
    p.lse_in = lse;
    p.dloss = dloss;
    p.dx = dx;
    p.dw = dw;
    p.ws = static_cast<uint8_t*>(workspace);
    return run_lm(p, workspace_bytes, true, stream);
}

moe_status_t moe_lm_distill_fwd(const void* x, const void* w, const int32_t* teacher_ids, const float* teacher_logits,
                                float temperature, float* loss, float* lse, int64_t T, int32_t D, int32_t V, int32_t K,
                                void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    LmProblem p{};
    p.x = x;
    p.w = w;
    p.T = T;
    p.D = D;
    p.V = V;
    p.K = K;
    p.teacher_ids = teacher_ids;
    p.teacher_logits = teacher_logits;
    p.temperature = temperature;
    p.loss = loss;
    p.lse = lse;
    p.ws = static_cast<uint8_t*>(workspace);
    return run_lm(p, workspace_bytes, false, stream);
}

moe_status_t moe_lm_distill_bwd(const void* x, const void* w, const int32_t* teacher_ids, const float* teacher_logits,
                                float temperature, const float* lse, const float* dloss, void* dx, void* dw, int64_t T,
                                int32_t D, int32_t V, int32_t K, void* workspace, size_t workspace_bytes,
                                moe_stream_t stream) {
    LmProblem p{};
    p.x = x;
    p.w = w;
    p.T = T;
    p.D = D;
    p.V = V;
    p.K = K;
    p.teacher_ids = teacher_ids;
    p.teacher_logits = teacher_logits;
    p.temperature = temperature;
    p.lse_in = lse;
    p.dloss = dloss;
    p.dx = dx;
    p.dw = dw;
    p.ws = static_cast<uint8_t*>(workspace);
    return run_lm(p, workspace_bytes, true, stream);
}

}  // extern "C"
