// block_norm_bwd.cu -- the way back through the norms after and before a block, its gate and the residual's scale.
//
//   hat = stream pre_rstd,  da = dstream + pre_rstd (dnormed pre_gamma - hat mean_d(dnormed pre_gamma hat))
//   dresidual = residual_scale da,  dpre_gamma = sum_t dnormed hat
//   bh = block post_rstd,  dgate = da bh post_gamma  (summed over t for a channel gate)
//   dpost_gamma = sum_t da gate bh,  gb = da gate post_gamma
//   dblock = post_rstd (gb - bh mean_d(gb bh))       (without a norm after the block: dblock = da gate)
//
// Bound by memory: 4 T D read and 2 T D written (a gate per token adds one of each; without norm and gate after
// the block, the block is not read). All sums are fp32, in a fixed order.
//
// Rows go through a ring in shared memory, one at a time through the two sums, of which the second needs the first.
// There are only two sums over the tokens, whatever is asked for: of dnormed hat, and of da bh (times a gate per
// token), from which a channel gate's and post_gamma's gradients follow by a factor per channel. They stay in
// registers; each block writes one row of them, and a second kernel adds the rows in block order.
#include <algorithm>

#include "row_ring.cuh"

namespace moe {
namespace {

struct BwdArgs {
    Param post_gamma, channel_gate, pre_gamma;
    const float *post_rstd, *pre_rstd;
    float* partial;  // [grid][2][D], or null
    int64_t rows;
    int32_t D;
    float scale;
};

template <typename T>
struct BwdRows {
    const T *dstream, *dnormed, *block, *stream, *gate;  // dstream, block and gate may be null
    T *dblock, *dresidual, *dgate;                       // dgate: per token, or null
};

// Twelve tensors' rows in the ring: four stages of the three that there always may be, three of four, two of five.
constexpr int kBwdTensors = 12;
template <typename T>
constexpr int kBwdSmem = kBwdTensors * kTensorBytes<T, kBnN<T>>;

template <typename T, int kGroup, bool kAligned>
__global__ void __launch_bounds__(kLnThreads, 1) k_bn_bwd(const BwdRows<T> x, const BwdArgs a) {
    constexpr int kN = kBnN<T>;
    using R = Row<T, kGroup, kAligned, kN>;
    constexpr int kVec = R::kVec, kVecs = R::kVecs, kRows = kLnThreads / kGroup, kTensor = kTensorBytes<T, kN>;
    using P = Pack<T, kVec>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[2][1][kLnThreads / 32];
    GroupSum<kGroup, 1> sum{buf};
    const int lane = threadIdx.x % kGroup;
    const int32_t D = a.D;
    const int64_t rows = a.rows, stride = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup;
    // the tensors' places in a stage
    const int at_ds = 2 * kTensor, at_b = at_ds + (x.dstream ? kTensor : 0), at_g = at_b + (x.block ? kTensor : 0);
    const int stage = at_g + (x.gate ? kTensor : 0);
    const int stages = stage <= 3 * kTensor ? 4 : stage <= 4 * kTensor ? 3 : 2;
    griddep_wait();
    griddep_launch_dependents();
    auto fetch = [&](int slot, int64_t r) {
        if (r < rows) {
            uint8_t* to = ring + slot * stage;
            R::fetch(to, x.dnormed, r, rows, D, lane);
            R::fetch(to + kTensor, x.stream, r, rows, D, lane);
            if (x.dstream) R::fetch(to + at_ds, x.dstream, r, rows, D, lane);
            if (x.block) R::fetch(to + at_b, x.block, r, rows, D, lane);
            if (x.gate) R::fetch(to + at_g, x.gate, r, rows, D, lane);
        }
        copy_commit();
    };
#pragma unroll 1
    for (int s = 0; s < stages - 1; ++s) fetch(s, row + s * stride);
    float pre[kN], post[kN], dpre[kN], dpost[kN];
    load_params<R>(a.pre_gamma, D, lane, 1.0f, pre);
    {
        float t[kN];
        load_params<R>(a.post_gamma, D, lane, 1.0f, post);
        load_params<R>(a.channel_gate, D, lane, 1.0f, t);
#pragma unroll
        for (int i = 0; i < kN; ++i) post[i] *= t[i], dpre[i] = 0.0f, dpost[i] = 0.0f;
    }
    const float inv_d = 1.0f / static_cast<float>(D);
    float next_pre = row < rows ? __ldg(a.pre_rstd + row) : 0.0f;
    float next_post = row < rows && a.post_rstd ? __ldg(a.post_rstd + row) : 1.0f;
    int slot = 0;
    for (; row < rows; row += stride) {
        const float pre_rstd = next_pre, post_rstd = next_post;
        if (row + stride < rows) {
            next_pre = __ldg(a.pre_rstd + row + stride);
            if (a.post_rstd) next_post = __ldg(a.post_rstd + row + stride);
        }
        if (stages == 4) copy_wait<2>();
        else if (stages == 3) copy_wait<1>();
        else copy_wait<0>();
        if constexpr (!kAligned) {  // the rows were copied by the whole group
            if constexpr (kGroup > 32) group_barrier(1 + threadIdx.x / kGroup, kGroup);
            else __syncwarp();
        }
        fetch(slot == 0 ? stages - 1 : slot - 1, row + (stages - 1) * stride);  // the place read in the last round
        const uint8_t* at = ring + slot * stage;
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (R::index(i, lane) < D) {
                const P pn = R::get(at, x.dnormed, row, D, i, lane), ps = R::get(at + kTensor, x.stream, row, D, i, lane);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const int n = i * kVec + e;
                    const float t = to_float(pn.v[e]) * (to_float(ps.v[e]) * pre_rstd);
                    dpre[n] += t;
                    s[0] = fmaf(t, pre[n], s[0]);
                }
            }
        }
        sum(s);
        const float m1 = s[0] * inv_d;
        float gb[kN];
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = R::index(i, lane);
            if (j < D) {
                const P pn = R::get(at, x.dnormed, row, D, i, lane), ps = R::get(at + kTensor, x.stream, row, D, i, lane);
                P pd, pb, pg, pr, pdg;
                if (x.dstream) pd = R::get(at + at_ds, x.dstream, row, D, i, lane);
                if (x.block) pb = R::get(at + at_b, x.block, row, D, i, lane);
                if (x.gate) pg = R::get(at + at_g, x.gate, row, D, i, lane);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const int n = i * kVec + e;
                    const float hat = to_float(ps.v[e]) * pre_rstd;
                    const float da = fmaf(pre_rstd, fmaf(-hat, m1, to_float(pn.v[e]) * pre[n]),
                                          x.dstream ? to_float(pd.v[e]) : 0.0f);
                    pr.v[e] = from_float<T>(a.scale * da);
                    float g = da;
                    const float bh = x.block ? to_float(pb.v[e]) * post_rstd : 0.0f;
                    if (x.gate) {
                        pdg.v[e] = from_float<T>(da * (bh * post[n]));
                        g *= to_float(pg.v[e]);
                    }
                    dpost[n] = fmaf(g, bh, dpost[n]);
                    gb[n] = g * post[n];
                    s[0] = fmaf(gb[n], bh, s[0]);
                }
                *reinterpret_cast<P*>(x.dresidual + row * D + j) = pr;
                if (x.gate && x.dgate) *reinterpret_cast<P*>(x.dgate + row * D + j) = pdg;
            }
        }
        float m2 = 0.0f;
        if (a.post_rstd) {
            sum(s);
            m2 = s[0] * inv_d;
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = R::index(i, lane);
            if (j < D) {
                P pb, pd;
                if (x.block) pb = R::get(at + at_b, x.block, row, D, i, lane);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float bh = x.block ? to_float(pb.v[e]) * post_rstd : 0.0f;
                    pd.v[e] = from_float<T>(post_rstd * fmaf(-bh, m2, gb[i * kVec + e]));
                }
                *reinterpret_cast<P*>(x.dblock + row * D + j) = pd;
            }
        }
        slot = slot + 1 == stages ? 0 : slot + 1;
    }
    if (a.partial == nullptr) return;
    // the block's row of partial sums: its groups own the same columns, and meet in the ring in group order
    float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * D;
    copy_wait<0>();
    __syncthreads();
    float* acc = reinterpret_cast<float*>(ring);  // [kRows][2][kGroup * kN]
    static_assert(kBwdSmem<T> >= 2 * kLnThreads * kN * 4, "the sums fit the ring");
    constexpr int kCols = kGroup * kN;
    float* own = acc + (threadIdx.x / kGroup) * 2 * kCols;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            own[R::index(i, lane) + e] = dpre[i * kVec + e];
            own[kCols + R::index(i, lane) + e] = dpost[i * kVec + e];
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += kLnThreads) {
        float p = 0.0f, q = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) p += acc[2 * r * kCols + j], q += acc[(2 * r + 1) * kCols + j];
        mine[j] = p;
        mine[D + j] = q;
    }
}

// Rows longer than a group holds: three passes over each of a block's rows, the second and third mostly from L2.
// The columns' sums are in shared memory where they fit, else in the block's row of partial sums; a column belongs
// to one thread.
constexpr int kLongSums = 96 * 1024;  // bytes of them in shared memory: two blocks share an SM
template <typename T, int kVec>
__global__ void __launch_bounds__(kLnThreads, 2) k_bn_bwd_long(const BwdRows<T> x, const BwdArgs a) {
    using P = Pack<T, kVec>;
    extern __shared__ __align__(16) float held[];
    __shared__ float buf[2][1][kLnThreads / 32];
    GroupSum<kLnThreads, 1> sum{buf};
    griddep_wait();
    griddep_launch_dependents();
    const int32_t D = a.D;
    const float inv_d = 1.0f / static_cast<float>(D);
    float* mine = a.partial ? a.partial + static_cast<int64_t>(blockIdx.x) * 2 * D : nullptr;
    float* sums = 2 * static_cast<int64_t>(D) * 4 <= kLongSums ? held : mine;
    if (mine)
        for (int j = threadIdx.x * kVec; j < D; j += kLnThreads * kVec)
#pragma unroll
            for (int e = 0; e < kVec; ++e) sums[j + e] = 0.0f, sums[D + j + e] = 0.0f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * D;
        const float pre_rstd = a.pre_rstd[row], post_rstd = a.post_rstd ? a.post_rstd[row] : 1.0f;
        auto get = [&](const T* p, int j) { return *reinterpret_cast<const P*>(p + at + j); };
        float s[1] = {0.0f};
#pragma unroll 2
        for (int j = threadIdx.x * kVec; j < D; j += kLnThreads * kVec) {
            const P pn = get(x.dnormed, j), ps = get(x.stream, j);
            float g[kVec];
            load_param<kVec>(a.pre_gamma, j, 1.0f, g);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float t = to_float(pn.v[e]) * (to_float(ps.v[e]) * pre_rstd);
                if (mine) sums[j + e] += t;
                s[0] = fmaf(t, g[e], s[0]);
            }
        }
        sum(s);
        const float m1 = s[0] * inv_d;
        // da and what comes after it, for the second sum and again for the outputs
        auto back = [&](int j, float (&da)[kVec], float (&bh)[kVec], float (&g)[kVec], float (&w)[kVec]) {
            const P pn = get(x.dnormed, j), ps = get(x.stream, j);
            P pd, pb, pg;
            if (x.dstream) pd = get(x.dstream, j);
            if (x.block) pb = get(x.block, j);
            if (x.gate) pg = get(x.gate, j);
            float pre[kVec], c[kVec];
            load_param<kVec>(a.pre_gamma, j, 1.0f, pre);
            load_param<kVec>(a.post_gamma, j, 1.0f, w);
            load_param<kVec>(a.channel_gate, j, 1.0f, c);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float hat = to_float(ps.v[e]) * pre_rstd;
                da[e] = fmaf(pre_rstd, fmaf(-hat, m1, to_float(pn.v[e]) * pre[e]), x.dstream ? to_float(pd.v[e]) : 0.0f);
                bh[e] = x.block ? to_float(pb.v[e]) * post_rstd : 0.0f;
                g[e] = x.gate ? da[e] * to_float(pg.v[e]) : da[e];
                w[e] *= c[e];
            }
        };
        float m2 = 0.0f;
        if (a.post_rstd) {
            s[0] = 0.0f;
#pragma unroll 2
            for (int j = threadIdx.x * kVec; j < D; j += kLnThreads * kVec) {
                float da[kVec], bh[kVec], g[kVec], w[kVec];
                back(j, da, bh, g, w);
#pragma unroll
                for (int e = 0; e < kVec; ++e) s[0] = fmaf(g[e] * w[e], bh[e], s[0]);
            }
            sum(s);
            m2 = s[0] * inv_d;
        }
        for (int j = threadIdx.x * kVec; j < D; j += kLnThreads * kVec) {
            float da[kVec], bh[kVec], g[kVec], w[kVec];
            back(j, da, bh, g, w);
            P pr, pd, pdg;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                pr.v[e] = from_float<T>(a.scale * da[e]);
                pdg.v[e] = from_float<T>(da[e] * (bh[e] * w[e]));
                pd.v[e] = from_float<T>(post_rstd * fmaf(-bh[e], m2, g[e] * w[e]));
                if (mine) sums[D + j + e] = fmaf(g[e], bh[e], sums[D + j + e]);
            }
            *reinterpret_cast<P*>(x.dresidual + at + j) = pr;
            *reinterpret_cast<P*>(x.dblock + at + j) = pd;
            if (x.gate && x.dgate) *reinterpret_cast<P*>(x.dgate + at + j) = pdg;
        }
    }
    if (mine && sums != mine)
        for (int j = threadIdx.x * kVec; j < D; j += kLnThreads * kVec)
#pragma unroll
            for (int e = 0; e < kVec; ++e) mine[j + e] = sums[j + e], mine[D + j + e] = sums[D + j + e];
}

// The blocks' rows of partial sums in block order, and from them the parameters' gradients. A block owns 32 columns
// of one of the two sums; its warps take the rows in turn and meet in shared memory.
constexpr int kGradWarps = 16;
struct GradArgs {
    const float* partial;
    Param post_gamma, channel_gate;
    int32_t blocks, D, param_dtype;
    void *dpre_gamma, *dpost_gamma, *dgate;  // dgate: of a channel gate
};
__global__ void __launch_bounds__(32 * kGradWarps) k_bn_param_grads(const GradArgs a) {
    __shared__ float acc[kGradWarps][32];
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.y == 0 ? a.dpre_gamma == nullptr : a.dpost_gamma == nullptr && a.dgate == nullptr) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + lane;
    constexpr int kEach = (kBnMaxBlocks + kGradWarps - 1) / kGradWarps;
    float v[kEach], s = 0.0f;  // all of a warp's rows at once: one latency instead of one per row
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int b = warp + u * kGradWarps;
        v[u] = j < a.D && b < a.blocks ? a.partial[(static_cast<int64_t>(b) * 2 + blockIdx.y) * a.D + j] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) s += v[u];
    acc[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || j >= a.D) return;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kGradWarps; ++w) s += acc[w][lane];
    if (blockIdx.y == 0) {
        store_param(a.dpre_gamma, a.param_dtype, j, s);
        return;
    }
    float g[1], c[1];
    load_param<1>(a.post_gamma, j, 1.0f, g);
    load_param<1>(a.channel_gate, j, 1.0f, c);
    if (a.dpost_gamma) store_param(a.dpost_gamma, a.param_dtype, j, s * c[0]);
    if (a.dgate) store_param(a.dgate, a.param_dtype, j, s * g[0]);
}

template <typename T, int kGroup, bool kAligned>
cudaError_t run(const BlockNormProblem& p, const BwdRows<T>& x, const BwdArgs& a, int* blocks, cudaStream_t stream) {
    const cudaError_t e = allow_smem<&k_bn_bwd<T, kGroup, kAligned>>(kBwdSmem<T>);
    if (e != cudaSuccess) return e;
    *blocks = static_cast<int>(std::min<int64_t>({ceil_div(p.T, kLnThreads / kGroup), p.sm_count, kBnMaxBlocks}));
    return launch_pdl(k_bn_bwd<T, kGroup, kAligned>, dim3(*blocks), dim3(kLnThreads), kBwdSmem<T>, stream, x, a);
}

template <typename T, bool kAligned>
cudaError_t dispatch(const BlockNormProblem& p, const BwdRows<T>& x, const BwdArgs& a, int* blocks, cudaStream_t stream) {
    constexpr int kN = kBnN<T>;
    if (p.D <= 32 * kN) return run<T, 32, kAligned>(p, x, a, blocks, stream);
    if (p.D <= 64 * kN) return run<T, 64, kAligned>(p, x, a, blocks, stream);
    if (p.D <= 128 * kN) return run<T, 128, kAligned>(p, x, a, blocks, stream);
    if (p.D <= 256 * kN) return run<T, 256, kAligned>(p, x, a, blocks, stream);
    if (p.D <= 512 * kN) return run<T, 512, kAligned>(p, x, a, blocks, stream);
    constexpr int kVec = kAligned ? 16 / static_cast<int>(sizeof(T)) : 1;
    const cudaError_t e = allow_smem<&k_bn_bwd_long<T, kVec>>(kLongSums);
    if (e != cudaSuccess) return e;
    const int64_t sums = 8 * static_cast<int64_t>(p.D);
    *blocks = static_cast<int>(std::min<int64_t>({p.T, 2 * p.sm_count, kBnMaxBlocks}));
    return launch_pdl(k_bn_bwd_long<T, kVec>, dim3(*blocks), dim3(kLnThreads),
                      static_cast<size_t>(a.partial && sums <= kLongSums ? sums : 0), stream, x, a);
}

template <typename T>
cudaError_t of_type(const BlockNormProblem& p, int* blocks, cudaStream_t stream) {
    const T* gate = p.gate_per_token ? static_cast<const T*>(p.gate) : nullptr;
    const bool needs_block = p.post_rstd_in || p.gate;
    const BwdRows<T> x{static_cast<const T*>(p.dstream), static_cast<const T*>(p.dnormed),
                       needs_block ? static_cast<const T*>(p.block) : nullptr, static_cast<const T*>(p.stream), gate,
                       static_cast<T*>(p.dblock), static_cast<T*>(p.dresidual),
                       gate ? static_cast<T*>(p.dgate) : nullptr};
    const BwdArgs a{param(p.post_gamma, p.param_dtype), param(gate ? nullptr : p.gate, p.param_dtype),
                    param(p.pre_gamma, p.param_dtype), p.post_rstd_in, p.pre_rstd_in, p.partial, p.T, p.D,
                    p.residual_scale};
    const int64_t bytes = static_cast<int64_t>(p.D) * sizeof(T);
    bool whole = true;
    for (const void* t : {static_cast<const void*>(x.dstream), static_cast<const void*>(x.dnormed),
                          static_cast<const void*>(x.block), static_cast<const void*>(x.stream),
                          static_cast<const void*>(x.gate), static_cast<const void*>(x.dblock),
                          static_cast<const void*>(x.dresidual), static_cast<const void*>(x.dgate)})
        whole = whole && rows_aligned16(t, bytes);
    return whole ? dispatch<T, true>(p, x, a, blocks, stream) : dispatch<T, false>(p, x, a, blocks, stream);
}

}  // namespace

moe_status_t launch_block_norm_bwd(const BlockNormProblem& in, cudaStream_t stream) {
    BlockNormProblem p = in;
    const bool channel_grad = p.dgate && !p.gate_per_token;
    if (!p.dpre_gamma && !p.dpost_gamma && !channel_grad) p.partial = nullptr;
    int blocks = 0;
    cudaError_t e = p.dtype == MOE_DTYPE_F32    ? of_type<float>(p, &blocks, stream)
                    : p.dtype == MOE_DTYPE_BF16 ? of_type<__nv_bfloat16>(p, &blocks, stream)
                                                : of_type<__half>(p, &blocks, stream);
    if (e == cudaSuccess && p.partial) {
        const GradArgs g{p.partial, param(p.post_gamma, p.param_dtype),
                         param(p.gate_per_token ? nullptr : p.gate, p.param_dtype), blocks, p.D, p.param_dtype,
                         p.dpre_gamma, p.dpost_gamma, channel_grad ? p.dgate : nullptr};
        e = launch_pdl(k_bn_param_grads, dim3(static_cast<unsigned>(ceil_div(p.D, 32)), 2), dim3(32 * kGradWarps), 0,
                       stream, g);
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
