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
//
// Measured (calls in a graph; in brackets the bytes at the copy rate): 16384 x 7168 bf16 275 us (208), with a gate per
// token 339 us (277), 4096 x 2048 without a norm after the block 20 us (12), 16384 x 7001 359 us (203), 8192 x 7168 f32
// 373 us (208). Bound by the two dependent sums of a row where it is not the memory: issue is 50 %, and 118 to 128
// registers (16 of the 16-bit kernels spill 4 to 16 bytes) leave no room for a second row. Without a norm or a gate after
// the block there is one sum and 102 registers, and one row at a time all the same. Blocks of 1024 threads took 325 us
// against 270, one reduction for both sums the same. The kernel for long rows of 16-bit types spills 224 to 344 bytes at the
// 64 registers that two blocks to an SM leave.
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
    int tensor, stages;  // the ring: bytes of a tensor's row, and stages
};

template <typename T>
struct BwdRows {
    const T *dstream, *dnormed, *block, *stream, *gate;  // dstream, block and gate may be null
    T *dblock, *dresidual, *dgate;                       // dgate: per token, or null
};

// The ring: up to four stages of the three to five tensors, at least two.
constexpr int kBwdSmem = 224 * 1024;

// What there is of the block's side: nothing (its gradient is da alone), the block, the block and a gate per token.
enum Side { kNoBlock, kBlock, kTokenGate };

template <typename T, int kGroup, bool kWhole, Side kSide>
__global__ void __launch_bounds__(kLnThreads, 1) k_bn_bwd(const BwdRows<T> x, const BwdArgs a) {
    constexpr int kN = kBnN<T>;
    using C = Cells<T, kGroup, kWhole, kN>;
    using Pairs = typename C::Pairs;
    constexpr int kP = C::kPairs, kRows = kLnThreads / kGroup;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[2][1][kLnThreads / 32];
    GroupSum<kGroup, 1> sum{buf};
    const int lane = threadIdx.x % kGroup;
    const int32_t D = a.D;
    const int64_t rows = a.rows, stride = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup;
    const C cells(x.dnormed, row, D, lane);
    // the tensors' places in a stage: dnormed, stream, block, gate, dstream
    const int stream_at = a.tensor, block_at = 2 * a.tensor, gate_at = 3 * a.tensor;
    const int dstream_at = (kSide == kNoBlock ? 2 : kSide == kBlock ? 3 : 4) * a.tensor;
    const int stage = dstream_at + (x.dstream ? a.tensor : 0);
    auto fetch = [&](int slot, int64_t r) {
        if (r < rows) {
            uint8_t* to = ring + slot * stage;
            cells.fetch(to, x.dnormed, r, rows);
            cells.fetch(to + stream_at, x.stream, r, rows);
            if constexpr (kSide != kNoBlock) cells.fetch(to + block_at, x.block, r, rows);
            if constexpr (kSide == kTokenGate) cells.fetch(to + gate_at, x.gate, r, rows);
            if (x.dstream) cells.fetch(to + dstream_at, x.dstream, r, rows);
        }
        copy_commit();
    };
    griddep_wait();
    griddep_launch_dependents();
#pragma unroll 1
    for (int s = 0; s < a.stages - 1; ++s) fetch(s, row + s * stride);
    float2 pre[kN / 2], post[kN / 2], dpre[kN / 2], dpost[kN / 2];
    cells.params(a.pre_gamma, 1.0f, pre);
    cells.params(a.post_gamma, 1.0f, post);
    cells.params(a.channel_gate, 1.0f, dpost);
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
        post[i] = __fmul2_rn(post[i], dpost[i]);
        dpre[i] = dpost[i] = both(0.0f);
    }
    const float inv_d = 1.0f / static_cast<float>(D);
    auto rstd_of = [&](const float* p, int64_t r) { return p && r < rows ? __ldg(p + r) : 1.0f; };
    float pre_next = rstd_of(a.pre_rstd, row), post_next = rstd_of(a.post_rstd, row);
    int slot = 0;
    for (; row < rows; row += stride) {
        const float2 pre_rstd = both(pre_next), post_rstd = both(post_next);
        pre_next = rstd_of(a.pre_rstd, row + stride);
        post_next = rstd_of(a.post_rstd, row + stride);
        if (a.stages == 4) copy_wait<2>();
        else if (a.stages == 3) copy_wait<1>();
        else copy_wait<0>();
        uint8_t* at = ring + slot * stage;
        if constexpr (!kWhole)
            for (int t = 0; t < stage; t += a.tensor) cells.trim(at + t);
        fetch(slot == 0 ? a.stages - 1 : slot - 1, row + (a.stages - 1) * stride);  // the place read in the last round
        float2 part = both(0.0f);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) {
            if (cells.any(c)) {
                Pairs n, t;
                cells.get(at, c, n);
                cells.get(at + stream_at, c, t);
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    const float2 v = __fmul2_rn(n[i], __fmul2_rn(t[i], pre_rstd));
                    dpre[c * kP + i] = __fadd2_rn(dpre[c * kP + i], v);
                    part = __ffma2_rn(v, pre[c * kP + i], part);
                }
            }
        }
        float s[1] = {part.x + part.y};
        sum(s);
        const float2 m1 = both(-s[0] * inv_d);
        float2 gb[kN / 2];
        part = both(0.0f);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) {
            if (cells.any(c)) {
                Pairs n, t, d, b, g, out;
                cells.get(at, c, n);
                cells.get(at + stream_at, c, t);
                if (x.dstream) cells.get(at + dstream_at, c, d);
                if constexpr (kSide != kNoBlock) cells.get(at + block_at, c, b);
                if constexpr (kSide == kTokenGate) cells.get(at + gate_at, c, g);
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    const int k = c * kP + i;
                    float2 da = __ffma2_rn(__fmul2_rn(t[i], pre_rstd), m1, __fmul2_rn(n[i], pre[k]));
                    da = x.dstream ? __ffma2_rn(pre_rstd, da, d[i]) : __fmul2_rn(pre_rstd, da);
                    out[i] = __fmul2_rn(both(a.scale), da);
                    if constexpr (kSide != kNoBlock) {
                        const float2 bh = __fmul2_rn(b[i], post_rstd);
                        if constexpr (kSide == kTokenGate) {
                            b[i] = __fmul2_rn(da, __fmul2_rn(bh, post[k]));  // the gate's gradient
                            da = __fmul2_rn(da, g[i]);
                        }
                        dpost[k] = __ffma2_rn(da, bh, dpost[k]);
                        gb[k] = __fmul2_rn(da, post[k]);
                        part = __ffma2_rn(gb[k], bh, part);
                    } else {
                        n[i] = da;
                    }
                }
                cells.put(x.dresidual, row, c, out);
                if constexpr (kSide == kTokenGate)
                    if (x.dgate) cells.put(x.dgate, row, c, b);
                if constexpr (kSide == kNoBlock) cells.put(x.dblock, row, c, n);
            }
        }
        if constexpr (kSide != kNoBlock) {
            float2 m2 = both(0.0f);
            if (a.post_rstd) {
                s[0] = part.x + part.y;
                sum(s);
                m2 = both(-s[0] * inv_d);
            }
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                if (cells.any(c)) {
                    Pairs b, out;
                    cells.get(at + block_at, c, b);
#pragma unroll
                    for (int i = 0; i < kP; ++i)
                        out[i] = __fmul2_rn(post_rstd, __ffma2_rn(__fmul2_rn(b[i], post_rstd), m2, gb[c * kP + i]));
                    cells.put(x.dblock, row, c, out);
                }
            }
        }
        slot = slot + 1 == a.stages ? 0 : slot + 1;
    }
    if (a.partial == nullptr) return;
    // the block's row of partial sums: its groups own the same columns, and meet in the ring in group order
    float* mine = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * D;
    copy_wait<0>();
    __syncthreads();
    float* acc = reinterpret_cast<float*>(ring);  // [kRows][2][kGroup * kN]
    static_assert(kBwdSmem >= 2 * kLnThreads * kN * 4, "the sums fit the ring");
    constexpr int kCols = kGroup * kN;
    float* own = acc + (threadIdx.x / kGroup) * 2 * kCols;
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c) {
#pragma unroll
        for (int e = 0; e < C::kC; ++e) {
            const int n = c * C::kC + e;
            if (cells.has(c, e)) {
                own[cells.index(c, e)] = n % 2 ? dpre[n / 2].y : dpre[n / 2].x;
                own[kCols + cells.index(c, e)] = n % 2 ? dpost[n / 2].y : dpost[n / 2].x;
            }
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

// Rows longer than a group holds, and tensors that lie differently to 16-byte pieces: three passes over each of a
// block's rows, the second and third mostly from L2.
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

template <typename T, int kGroup, bool kWhole, Side kSide>
cudaError_t run_side(const BlockNormProblem& p, const BwdRows<T>& x, BwdArgs a, int* blocks, cudaStream_t stream) {
    const cudaError_t e = allow_smem<&k_bn_bwd<T, kGroup, kWhole, kSide>>(kBwdSmem);
    if (e != cudaSuccess) return e;
    *blocks = static_cast<int>(row_blocks(p.T, kLnThreads / kGroup, std::min(p.sm_count, kBnMaxBlocks)));
    const int tensors = (kSide == kNoBlock ? 2 : kSide == kBlock ? 3 : 4) + (x.dstream ? 1 : 0);
    a.tensor = tensor_stride<T, kGroup>(p.D);
    a.stages = std::min(4, kBwdSmem / (tensors * a.tensor));
    static_assert(2 * 5 * kTensorBytes<T, kBnN<T>> <= kBwdSmem, "two stages of everything");
    return launch_pdl(k_bn_bwd<T, kGroup, kWhole, kSide>, dim3(*blocks), dim3(kLnThreads), kBwdSmem, stream, x, a);
}

template <typename T, int kGroup, bool kWhole>
cudaError_t run(const BlockNormProblem& p, const BwdRows<T>& x, const BwdArgs& a, int* blocks, cudaStream_t stream) {
    if (x.gate) return run_side<T, kGroup, kWhole, kTokenGate>(p, x, a, blocks, stream);
    if (x.block) return run_side<T, kGroup, kWhole, kBlock>(p, x, a, blocks, stream);
    return run_side<T, kGroup, kWhole, kNoBlock>(p, x, a, blocks, stream);
}

template <typename T, bool kWhole>
cudaError_t dispatch(const BlockNormProblem& p, const BwdRows<T>& x, const BwdArgs& a, int* blocks, cudaStream_t stream) {
    constexpr int kN = kBnN<T>;
    const int32_t held = kWhole ? p.D : p.D + 16 / static_cast<int>(sizeof(T)) - 1;  // with what comes before the row
    if (held <= 32 * kN) return run<T, 32, kWhole>(p, x, a, blocks, stream);
    if (held <= 64 * kN) return run<T, 64, kWhole>(p, x, a, blocks, stream);
    if (held <= 128 * kN) return run<T, 128, kWhole>(p, x, a, blocks, stream);
    if (held <= 256 * kN) return run<T, 256, kWhole>(p, x, a, blocks, stream);
    return run<T, 512, kWhole>(p, x, a, blocks, stream);
}

template <typename T>
cudaError_t of_type(const BlockNormProblem& p, int* blocks, cudaStream_t stream) {
    constexpr int kC = 16 / static_cast<int>(sizeof(T));
    const T* gate = p.gate_per_token ? static_cast<const T*>(p.gate) : nullptr;
    const bool needs_block = p.post_rstd_in || p.gate;
    const BwdRows<T> x{static_cast<const T*>(p.dstream), static_cast<const T*>(p.dnormed),
                       needs_block ? static_cast<const T*>(p.block) : nullptr, static_cast<const T*>(p.stream), gate,
                       static_cast<T*>(p.dblock), static_cast<T*>(p.dresidual),
                       gate ? static_cast<T*>(p.dgate) : nullptr};
    const BwdArgs a{param(p.post_gamma, p.param_dtype), param(gate ? nullptr : p.gate, p.param_dtype),
                    param(p.pre_gamma, p.param_dtype), p.post_rstd_in, p.pre_rstd_in, p.partial, p.T, p.D,
                    p.residual_scale, 0, 0};
    const bool alike = lie_alike({x.dstream, x.dnormed, x.block, x.stream, x.gate, x.dblock, x.dresidual, x.dgate});
    const bool whole = alike && rows_aligned16(x.dnormed, static_cast<int64_t>(p.D) * sizeof(T));
    if (whole && p.D <= kBnMaxHeldD<T>) return dispatch<T, true>(p, x, a, blocks, stream);
    if (alike && !whole && p.D + kC - 1 <= kBnMaxHeldD<T>) return dispatch<T, false>(p, x, a, blocks, stream);
    const int64_t sums = 8 * static_cast<int64_t>(p.D);
    *blocks = static_cast<int>(std::min<int64_t>({p.T, 2 * p.sm_count, kBnMaxBlocks}));
    auto go = [&](auto kernel, cudaError_t allowed) {
        if (allowed != cudaSuccess) return allowed;
        return launch_pdl(kernel, dim3(*blocks), dim3(kLnThreads),
                          static_cast<size_t>(a.partial && sums <= kLongSums ? sums : 0), stream, x, a);
    };
    return whole ? go(k_bn_bwd_long<T, kC>, allow_smem<&k_bn_bwd_long<T, kC>>(kLongSums))
                 : go(k_bn_bwd_long<T, 1>, allow_smem<&k_bn_bwd_long<T, 1>>(kLongSums));
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
