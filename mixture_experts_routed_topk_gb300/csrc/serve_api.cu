// serve_api.cu -- the C ABI of the operators of a decoding step: argument checks, then the launches. As in
// moe_api.cu, the checks that need no GPU run first, and an entry point only enqueues work on the caller's
// stream.
#include <cuda_runtime.h>

#include "serve_internal.cuh"

namespace moe {
namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The shape limits of the layer for a few tokens.
moe_status_t check_few(int64_t T, int32_t D, int32_t F, int32_t E, int32_t K) {
    if (T < 0 || D <= 0 || F <= 0 || E <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || D % 64 != 0 || F % 64 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T > kFewMaxTokens || T * K > kFewMaxPairs) return MOE_ERR_UNSUPPORTED_SHAPE;
    // rows of weights and tile numbers are 32-bit
    if (static_cast<int64_t>(E) * 2 * F >= (int64_t{1} << 31) || static_cast<int64_t>(E) * D >= (int64_t{1} << 31))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// The status word, and H [T K, F] in two bf16 parts.
size_t few_workspace(int64_t T, int32_t F, int32_t K) {
    return kAlign + (4 * static_cast<size_t>(T) * K * F + kAlign - 1) / kAlign * kAlign;
}

// The checks that both entry points share; T = 0 returns before anything is looked at.
moe_status_t run_few(FewProblem& p, int64_t T, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    if (!p.x || !p.w13 || !p.w2 || !p.out || !workspace) return MOE_ERR_INVALID_ARG;
    if (!aligned(p.x, 16) || !aligned(p.w13, 16) || !aligned(p.w2, 16) || !aligned(p.out, 16) ||
        !aligned(workspace, kAlign))
        return MOE_ERR_MISALIGNED;
    if (workspace_bytes < few_workspace(T, p.F, p.K)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    DeviceInfo dev;
    const moe_status_t st = device_info(&dev);
    if (st != MOE_OK) return st;
    if (!dev.supported) return MOE_ERR_UNSUPPORTED_DEVICE;
    p.T = static_cast<int32_t>(T);
    p.status = static_cast<uint32_t*>(workspace);
    p.h = static_cast<uint8_t*>(workspace) + kAlign;
    p.sm_count = dev.sm_count;
    return launch_few(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_few_workspace_bytes(int64_t T, int32_t D, int32_t F, int32_t E, int32_t K) {
    if (T == 0 || check_few(T, D, F, E, K) != MOE_OK) return 0;
    return few_workspace(T, F, K);
}

moe_status_t moe_routed_experts_fwd_few(const void* x, const int32_t* topk_ids, const void* topk_scores,
                                        int32_t scores_dtype, const void* w13, const void* w2, void* out, int64_t T,
                                        int32_t D, int32_t F, int32_t E, int32_t K, void* workspace,
                                        size_t workspace_bytes, moe_stream_t stream) {
    if (scores_dtype != MOE_SCORES_F32 && scores_dtype != MOE_SCORES_BF16) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_few(T, D, F, E, K);
    if (st != MOE_OK || T == 0) return st;
    if (!topk_ids || !topk_scores) return MOE_ERR_INVALID_ARG;
    if (!aligned(topk_ids, 16) || !aligned(topk_scores, 16)) return MOE_ERR_MISALIGNED;
    FewProblem p{};
    p.x = x;
    p.ids = topk_ids;
    p.scores = topk_scores;
    p.scores_dtype = scores_dtype;
    p.w13 = w13;
    p.w2 = w2;
    p.out = out;
    p.D = D;
    p.F = F;
    p.E = E;
    p.K = K;
    return run_few(p, T, workspace, workspace_bytes, stream);
}

moe_status_t moe_layer_fwd_few(const void* x, const void* logits, int32_t dtype, int32_t normalize, const void* w13,
                               const void* w2, int32_t* topk_ids, float* topk_scores, void* out, int64_t T, int32_t D,
                               int32_t F, int32_t E, int32_t K, void* workspace, size_t workspace_bytes,
                               moe_stream_t stream) {
    if ((dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) || K > E) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_few(T, D, F, E, K);
    if (st != MOE_OK || T == 0) return st;
    if (!logits || !topk_ids || !topk_scores) return MOE_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == MOE_DTYPE_F32 ? 4 : 2) || !aligned(topk_ids, 16) || !aligned(topk_scores, 16))
        return MOE_ERR_MISALIGNED;
    FewProblem p{};
    p.x = x;
    p.logits = logits;
    p.logits_dtype = dtype;
    p.normalize = normalize != 0;
    p.ids_out = topk_ids;
    p.scores_out = topk_scores;
    p.w13 = w13;
    p.w2 = w2;
    p.out = out;
    p.D = D;
    p.F = F;
    p.E = E;
    p.K = K;
    return run_few(p, T, workspace, workspace_bytes, stream);
}

moe_status_t moe_sample(const void* logits, int32_t dtype, const float* uniform, const float* temperature,
                        const int32_t* top_k, const float* top_p, const float* min_p, int32_t* token, float* logprob,
                        int64_t T, int32_t V, moe_stream_t stream) {
    if ((dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) || T < 0 || V <= 0)
        return MOE_ERR_INVALID_ARG;
    if (T >= (int64_t{1} << 31) || V > kSampleMaxV) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !uniform || !token) return MOE_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == MOE_DTYPE_F32 ? 4 : 2) || !aligned(uniform, 4) || !aligned(temperature, 4) ||
        !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(token, 4) || !aligned(logprob, 4))
        return MOE_ERR_MISALIGNED;
    DeviceInfo dev;
    const moe_status_t st = device_info(&dev);
    if (st != MOE_OK) return st;
    if (!dev.supported) return MOE_ERR_UNSUPPORTED_DEVICE;
    const SampleProblem p{logits, dtype, uniform, temperature, top_k, top_p, min_p, token, logprob, T, V, dev.sm_count};
    return launch_sample(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
