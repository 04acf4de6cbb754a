// block_norm_fwd.cu -- the norms after and before a block, with its gate and the residual's scale, in one pass.
//
//   u      = block post_rstd post_gamma,  post_rstd = 1 / sqrt(mean_d(block^2) + eps)   (or u = block)
//   stream = residual_scale residual + gate u
//   normed = stream pre_rstd pre_gamma,   pre_rstd = 1 / sqrt(mean_d(stream^2) + eps)
//
// Bound by memory: block and residual (and a gate per token) are read once, stream and normed written once,
// 4 T D elements where four separate kernels move 9. The second norm takes the sum before it is rounded. All
// arithmetic is fp32.
//
// Rows go through a ring in shared memory as the layer norm's do, two at a time through the two sums (the second
// needs the first row's scale), with the products of the constant factors in registers: post_gamma times a
// channel gate, and pre_gamma. Rows longer than a group holds are read three times, mostly from L2.
//
// Measured (calls in a graph; in brackets the bytes at the copy rate): 16384 x 7168 bf16 145 us (139), 16 rows 4.4 us,
// 16384 x 512 14 us (10), 8191 x 1001 f16 with a gate per token 23 us (12), 16384 x 7001 bf16 193 us (135: rows on no
// 16-byte boundary, where every piece is looked at for elements of the neighbours before it is used and before it is
// written), 8192 x 7168 f32 219 us (139: three readings).
#include <algorithm>

#include "row_ring.cuh"

namespace moe {
namespace {

struct FwdArgs {
    Param post_gamma, channel_gate, pre_gamma;
    float *post_rstd, *pre_rstd;
    int64_t rows;
    int32_t D;
    float scale, eps;
};

// Two rows at a time; the ring has six stages of two tensors, or four of three: 200 KB.
constexpr int kBatch = 2;
template <typename T>
constexpr int kFwdSmem = 12 * kTensorBytes<T, kBnN<T>>;

// The pointers are not declared restrict: stream may be residual or block, normed too.
template <typename T, int kGroup, bool kWhole>
__global__ void __launch_bounds__(kLnThreads, 1)
    k_bn_fwd(const T* block, const T* residual, const T* gate, T* stream, T* normed, const FwdArgs a) {
    constexpr int kN = kBnN<T>;
    using C = Cells<T, kGroup, kWhole, kN>;
    using Pairs = typename C::Pairs;
    constexpr int kP = C::kPairs, kRows = kLnThreads / kGroup, kTensor = kTensorBytes<T, kN>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[2][kBatch][kLnThreads / 32];
    GroupSum<kGroup, kBatch> sum{buf};
    const int lane = threadIdx.x % kGroup;
    const int32_t D = a.D;
    const int64_t rows = a.rows, stride = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup;
    const C cells(block, row, D, lane);
    const int tensors = gate ? 3 : 2, stages = gate ? 4 : 6, stage = tensors * kTensor;
    griddep_wait();
    griddep_launch_dependents();
    auto fetch = [&](int slot, int64_t r) {
        if (r < rows) {
            uint8_t* to = ring + slot * stage;
            cells.fetch(to, block, r, rows);
            cells.fetch(to + kTensor, residual, r, rows);
            if (gate) cells.fetch(to + 2 * kTensor, gate, r, rows);
        }
        copy_commit();
    };
#pragma unroll 1
    for (int s = 0; s < stages - kBatch; ++s) fetch(s, row + s * stride);
    float2 post[kN / 2], pre[kN / 2];
    cells.params(a.post_gamma, 1.0f, post);
    cells.params(a.channel_gate, 1.0f, pre);
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) post[i] = __fmul2_rn(post[i], pre[i]);
    cells.params(a.pre_gamma, 1.0f, pre);
    const float inv_d = 1.0f / static_cast<float>(D);
    int slot = 0;
    for (; row < rows; row += kBatch * stride) {
        if (gate) copy_wait<0>();
        else copy_wait<2>();
        if constexpr (!kWhole) {
            for (int t = 0; t < tensors; ++t)
#pragma unroll
                for (int k = 0; k < kBatch; ++k) cells.trim(ring + (slot + k) * stage + t * kTensor);
        }
        const int last = slot == 0 ? stages - kBatch : slot - kBatch;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) fetch(last + k, row + (stages - kBatch + k) * stride);
        float2 v[kBatch][kN / 2], part[kBatch];
        float s[kBatch], rstd[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            part[k] = both(0.0f);
            rstd[k] = 1.0f;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                Pairs b;
                if (row + k * stride < rows && cells.any(c)) {
                    cells.get(ring + (slot + k) * stage, c, b);
                } else {
#pragma unroll
                    for (int i = 0; i < kP; ++i) b[i] = both(0.0f);
                }
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    v[k][c * kP + i] = b[i];
                    part[k] = __ffma2_rn(b[i], b[i], part[k]);
                }
            }
            s[k] = part[k].x + part[k].y;
        }
        if (a.post_rstd) {
            sum(s);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                rstd[k] = 1.0f / sqrtf(s[k] * inv_d + a.eps);
                if (lane == 0 && row + k * stride < rows) a.post_rstd[row + k * stride] = rstd[k];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t r = row + k * stride;
            const uint8_t* at = ring + (slot + k) * stage;
            part[k] = both(0.0f);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                if (r < rows && cells.any(c)) {
                    Pairs t, g;
                    cells.get(at + kTensor, c, t);
                    if (gate) cells.get(at + 2 * kTensor, c, g);
#pragma unroll
                    for (int i = 0; i < kP; ++i) {
                        const int n = c * kP + i;
                        float2 u = __fmul2_rn(__fmul2_rn(v[k][n], both(rstd[k])), post[n]);
                        if (gate) u = __fmul2_rn(u, g[i]);
                        v[k][n] = __ffma2_rn(both(a.scale), t[i], u);
                        part[k] = __ffma2_rn(v[k][n], v[k][n], part[k]);
                    }
                }
            }
            s[k] = part[k].x + part[k].y;
        }
        sum(s);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t r = row + k * stride;
            if (r >= rows) break;
            const float pre_rstd = 1.0f / sqrtf(s[k] * inv_d + a.eps);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                if (cells.any(c)) {
                    Pairs t, n;
#pragma unroll
                    for (int i = 0; i < kP; ++i) {
                        t[i] = v[k][c * kP + i];
                        n[i] = __fmul2_rn(__fmul2_rn(t[i], both(pre_rstd)), pre[c * kP + i]);
                    }
                    cells.put(stream, r, c, t);
                    cells.put(normed, r, c, n);
                }
            }
            if (lane == 0) a.pre_rstd[r] = pre_rstd;
        }
        slot = slot + kBatch == stages ? 0 : slot + kBatch;
    }
}

// Rows longer than a group holds, and tensors that lie differently to 16-byte pieces: a block to each row, three
// passes.
template <typename T, int kVec>
__global__ void __launch_bounds__(kLnThreads)
    k_bn_fwd_long(const T* block, const T* residual, const T* gate, T* stream, T* normed, const FwdArgs a) {
    __shared__ float buf[2][1][kLnThreads / 32];
    GroupSum<kLnThreads, 1> sum{buf};
    griddep_wait();
    griddep_launch_dependents();
    const int32_t D = a.D;
    const int64_t row = blockIdx.x, at = row * D;
    const float inv_d = 1.0f / static_cast<float>(D);
    using P = Pack<T, kVec>;
    float s[1] = {0.0f}, rstd = 1.0f;
    if (a.post_rstd) {
#pragma unroll 2
        for (int j = threadIdx.x * kVec; j < D; j += kLnThreads * kVec) {
            const P p = *reinterpret_cast<const P*>(block + at + j);
#pragma unroll
            for (int e = 0; e < kVec; ++e) s[0] = fmaf(to_float(p.v[e]), to_float(p.v[e]), s[0]);
        }
        sum(s);
        rstd = 1.0f / sqrtf(s[0] * inv_d + a.eps);
        if (threadIdx.x == 0) a.post_rstd[row] = rstd;
    }
    auto combine = [&](int j, float (&u)[kVec]) {
        const P pb = *reinterpret_cast<const P*>(block + at + j), pr = *reinterpret_cast<const P*>(residual + at + j);
        float g[kVec], c[kVec];
        load_param<kVec>(a.post_gamma, j, 1.0f, g);
        load_param<kVec>(a.channel_gate, j, 1.0f, c);
        P pg;
        if (gate) pg = *reinterpret_cast<const P*>(gate + at + j);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            float t = to_float(pb.v[e]) * rstd * (g[e] * c[e]);
            if (gate) t *= to_float(pg.v[e]);
            u[e] = fmaf(a.scale, to_float(pr.v[e]), t);
        }
    };
    s[0] = 0.0f;
#pragma unroll 2
    for (int j = threadIdx.x * kVec; j < D; j += kLnThreads * kVec) {
        float u[kVec];
        combine(j, u);
#pragma unroll
        for (int e = 0; e < kVec; ++e) s[0] = fmaf(u[e], u[e], s[0]);
    }
    sum(s);
    const float pre_rstd = 1.0f / sqrtf(s[0] * inv_d + a.eps);
    if (threadIdx.x == 0) a.pre_rstd[row] = pre_rstd;
    for (int j = threadIdx.x * kVec; j < D; j += kLnThreads * kVec) {
        float u[kVec], g[kVec];
        combine(j, u);
        load_param<kVec>(a.pre_gamma, j, 1.0f, g);
        P ps, pn;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            ps.v[e] = from_float<T>(u[e]);
            pn.v[e] = from_float<T>(u[e] * pre_rstd * g[e]);
        }
        *reinterpret_cast<P*>(stream + at + j) = ps;
        *reinterpret_cast<P*>(normed + at + j) = pn;
    }
}

template <typename T, int kGroup, bool kWhole>
cudaError_t run(const BlockNormProblem& p, const FwdArgs& a, const T* gate, cudaStream_t stream) {
    const cudaError_t e = allow_smem<&k_bn_fwd<T, kGroup, kWhole>>(kFwdSmem<T>);
    if (e != cudaSuccess) return e;
    const int64_t blocks = row_blocks(p.T, kLnThreads / kGroup, p.sm_count);
    return launch_pdl(k_bn_fwd<T, kGroup, kWhole>, dim3(static_cast<unsigned>(blocks)), dim3(kLnThreads), kFwdSmem<T>,
                      stream, static_cast<const T*>(p.block), static_cast<const T*>(p.residual), gate,
                      static_cast<T*>(p.stream), static_cast<T*>(p.normed), a);
}

template <typename T, bool kWhole>
cudaError_t dispatch(const BlockNormProblem& p, const FwdArgs& a, const T* gate, cudaStream_t stream) {
    constexpr int kN = kBnN<T>;
    const int32_t held = kWhole ? p.D : p.D + 16 / static_cast<int>(sizeof(T)) - 1;  // with what comes before the row
    if (held <= 32 * kN) return run<T, 32, kWhole>(p, a, gate, stream);
    if (held <= 64 * kN) return run<T, 64, kWhole>(p, a, gate, stream);
    if (held <= 128 * kN) return run<T, 128, kWhole>(p, a, gate, stream);
    if (held <= 256 * kN) return run<T, 256, kWhole>(p, a, gate, stream);
    return run<T, 512, kWhole>(p, a, gate, stream);
}

template <typename T>
cudaError_t of_type(const BlockNormProblem& p, cudaStream_t stream) {
    const FwdArgs a{param(p.post_gamma, p.param_dtype), param(p.gate_per_token ? nullptr : p.gate, p.param_dtype),
                    param(p.pre_gamma, p.param_dtype), p.post_rstd, p.pre_rstd, p.T, p.D, p.residual_scale, p.eps};
    constexpr int kC = 16 / static_cast<int>(sizeof(T));
    const T* gate = p.gate_per_token ? static_cast<const T*>(p.gate) : nullptr;
    const bool alike = lie_alike({p.block, p.residual, p.stream, p.normed, gate});
    const bool whole = alike && rows_aligned16(p.block, static_cast<int64_t>(p.D) * sizeof(T));
    if (whole && p.D <= kBnMaxHeldD<T>) return dispatch<T, true>(p, a, gate, stream);
    if (alike && !whole && p.D + kC - 1 <= kBnMaxHeldD<T>) return dispatch<T, false>(p, a, gate, stream);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(static_cast<unsigned>(p.T)), dim3(kLnThreads), 0, stream,
                          static_cast<const T*>(p.block), static_cast<const T*>(p.residual), gate,
                          static_cast<T*>(p.stream), static_cast<T*>(p.normed), a);
    };
    return whole ? go(k_bn_fwd_long<T, kC>) : go(k_bn_fwd_long<T, 1>);
}

}  // namespace

moe_status_t launch_block_norm_fwd(const BlockNormProblem& p, cudaStream_t stream) {
    const cudaError_t e = p.dtype == MOE_DTYPE_F32    ? of_type<float>(p, stream)
                          : p.dtype == MOE_DTYPE_BF16 ? of_type<__nv_bfloat16>(p, stream)
                                                      : of_type<__half>(p, stream);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
