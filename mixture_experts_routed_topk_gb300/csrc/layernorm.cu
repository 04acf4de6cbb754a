// layernorm.cu -- layer norm over the last dimension, forward and backward.
//
//   mean = sum_d x / D,  rstd = 1 / sqrt(sum_d (x - mean)^2 / D + eps),  xhat = (x - mean) rstd
//   y = xhat gamma + beta
//   with g = dy gamma:  dx = rstd (g - mean_d(g) - xhat mean_d(g xhat))
//   dgamma = sum_t dy xhat,  dbeta = sum_t dy
//
// Both directions are bound by memory: forward T D read and written once, backward 2 T D read and
// T D written. All arithmetic is fp32; the variance is taken from the centred values, so a large mean
// does not cancel it away.
//
// Rows up to 8192 elements: persistent blocks of 512 threads, in groups of 32 to 512 threads that own
// one row at a time (16 elements per thread). A group asynchronously copies the rows it will need
// next into a ring in shared memory, so that loads are in flight while it waits in the two row sums; it
// takes two rows through those sums at a time, and keeps the parameters in registers. Where rows start on
// 16-byte boundaries a thread copies and reads only its own elements; otherwise the group copies the aligned
// 16-byte pieces that cover the row, and each thread picks out its elements.
//
// The backward blocks keep their column sums of dy xhat and dy in registers, so dgamma and dbeta cost
// no extra pass over x and dy. Each block writes one row of partial sums, and a second kernel adds the
// rows in block order: the result does not depend on the order in which blocks finish.
//
// Longer rows are read two or three times, mostly from L2.
//
// Measured (device time; the copy rate is 6.79 TB/s): bf16 16384 x 7168 forward 87 us (5.4 TB/s), backward
// 121 us (5.8 TB/s), both bound by instruction issue and the waits in the row sums as much as by memory
// (a block per row without the ring and with the parameters read anew: 157 and 265 us); 4096 x 2048 11 and
// 16 us and fp16 8191 x 1001 13 and 24 us, where a group has seven rows or fewer and the latency of a launch,
// of the first loads and of four rounds decides. Long rows, bf16 4096 x 16384: 90 us forward, and 712 us
// backward, whose column sums go through global memory for every row (39 and 59 us at the copy rate).
#include <algorithm>

#include "row_ring.cuh"

namespace moe {
namespace {

// Rows a group takes through its sums together, and rows in the ring: with two at a time, those two, the
// two being fetched into the places of the last two, and the ones in between. Some 50 KB in flight hide
// the memory's latency at full rate; the ring takes up to 200 KB of an SM's shared memory. fp32 rows of
// the backward pass are so long that three single ones fill it.
template <typename T, bool kBackward>
constexpr int kLnBatch = kBackward && sizeof(T) == 4 ? 1 : 2;
template <typename T, bool kBackward>
constexpr int kLnStages = kBackward ? (sizeof(T) == 4 ? 3 : 6) : (sizeof(T) == 4 ? 6 : 10);
template <typename T, bool kBackward>
constexpr int kLnSmemBytes = kLnStages<T, kBackward> * (kBackward ? 2 : 1) * kTensorBytes<T>;

// x and y are not declared restrict: y may be x itself. A group has its row in registers before it writes
// it, and of the neighbouring rows that its pieces touch it uses nothing.
template <typename T, int kGroup, bool kAligned>
__global__ void __launch_bounds__(kLnThreads, 1)
    k_ln_fwd(const T* x, const Param gamma, const Param beta, T* y, float* __restrict__ mean_out,
             float* __restrict__ rstd_out, int64_t rows, int32_t D, float eps) {
    using R = Row<T, kGroup, kAligned>;
    constexpr int kVec = R::kVec, kVecs = R::kVecs, kStages = kLnStages<T, false>, kBatch = kLnBatch<T, false>;
    static_assert(kBatch == 2, "two rows share a sum");
    constexpr int kRows = kLnThreads / kGroup;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[2][2][kLnThreads / 32];
    GroupSum<kGroup, 2> sum{buf};
    const int lane = threadIdx.x % kGroup;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup;
    griddep_wait();
    griddep_launch_dependents();
    auto fetch = [&](int slot, int64_t r) {
        if (r < rows) R::fetch(ring + slot * kTensorBytes<T>, x, r, rows, D, lane);
        copy_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - kBatch; ++s) fetch(s, row + s * stride);
    float g[kLnN], b[kLnN];
    load_params<R>(gamma, D, lane, 1.0f, g);
    load_params<R>(beta, D, lane, 0.0f, b);
    const float inv_d = 1.0f / static_cast<float>(D);
    // slots go round in pairs: this round's pair, and the last round's, which is filled again
    int slot = 0;
    for (; row < rows; row += kBatch * stride) {
        copy_wait<kStages - 2 * kBatch>();
        if constexpr (!kAligned) {  // the rows were copied by the whole group
            if constexpr (kGroup > 32) group_barrier(1 + threadIdx.x / kGroup, kGroup);
            else __syncwarp();
        }
        const int last = slot == 0 ? kStages - kBatch : slot - kBatch;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) fetch(last + k, row + (kStages - kBatch + k) * stride);
        float v[kBatch][kLnN], s[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool live = row + k * stride < rows;
            s[k] = 0.0f;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                if (live && R::index(i, lane) < D) {
                    const auto p = R::get(ring + (slot + k) * kTensorBytes<T>, x, row + k * stride, D, i, lane);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) v[k][i * kVec + e] = to_float(p.v[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < kVec; ++e) v[k][i * kVec + e] = 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < kLnN; ++i) s[k] += v[k][i];
        }
        sum(s);
        float mean[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            mean[k] = s[k] * inv_d;
            s[k] = 0.0f;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                if (R::index(i, lane) < D) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const float c = v[k][i * kVec + e] - mean[k];
                        v[k][i * kVec + e] = c;
                        s[k] += c * c;
                    }
                }
            }
        }
        sum(s);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t r = row + k * stride;
            if (r >= rows) break;
            const float rstd = 1.0f / sqrtf(s[k] * inv_d + eps);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int j = R::index(i, lane);
                if (j < D) {
                    Pack<T, kVec> p;
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const int n = i * kVec + e;
                        p.v[e] = from_float<T>(fmaf(v[k][n] * rstd, g[n], b[n]));
                    }
                    *reinterpret_cast<Pack<T, kVec>*>(y + r * D + j) = p;
                }
            }
            if (lane == 0) {
                mean_out[r] = mean[k];
                rstd_out[r] = rstd;
            }
        }
        slot = slot + kBatch == kStages ? 0 : slot + kBatch;
    }
}

// Rows longer than the registers hold: three passes over the row, the second and third from L2.
constexpr int kLongThreads = kLnThreads;
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    k_ln_fwd_long(const T* x, const Param gamma, const Param beta, T* y, float* __restrict__ mean_out,
                  float* __restrict__ rstd_out, int32_t D, float eps) {
    __shared__ float buf[2][2][kLnThreads / 32];
    GroupSum<kLongThreads, 2> sum{buf};
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* xr = x + row * D;
    const float inv_d = 1.0f / static_cast<float>(D);
    float s[2] = {0.0f, 0.0f};
    for (int j = threadIdx.x; j < D; j += kLongThreads) s[0] += to_float(xr[j]);
    sum(s);
    const float mean = s[0] * inv_d;
    s[0] = 0.0f;
    for (int j = threadIdx.x; j < D; j += kLongThreads) {
        const float c = to_float(xr[j]) - mean;
        s[0] += c * c;
    }
    sum(s);
    const float rstd = 1.0f / sqrtf(s[0] * inv_d + eps);
    for (int j = threadIdx.x; j < D; j += kLongThreads) {
        float g[1], b[1];
        load_param<1>(gamma, j, 1.0f, g);
        load_param<1>(beta, j, 0.0f, b);
        y[row * D + j] = from_float<T>(fmaf((to_float(xr[j]) - mean) * rstd, g[0], b[0]));
    }
    if (threadIdx.x == 0) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }
}

// partial: [grid][2][D], or null where neither parameter gradient is wanted. dx may be dy or x.
template <typename T, int kGroup, bool kAligned>
__global__ void __launch_bounds__(kLnThreads, 1)
    k_ln_bwd(const T* dy, const T* x, const Param gamma, const float* __restrict__ mean_in,
             const float* __restrict__ rstd_in, T* dx, int64_t rows, int32_t D, float* __restrict__ partial) {
    using R = Row<T, kGroup, kAligned>;
    constexpr int kVec = R::kVec, kVecs = R::kVecs, kStages = kLnStages<T, true>, kBatch = kLnBatch<T, true>;
    constexpr int kRows = kLnThreads / kGroup;
    constexpr int kStage = 2 * kTensorBytes<T>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[2][2 * kBatch][kLnThreads / 32];
    GroupSum<kGroup, 2 * kBatch> sum{buf};
    const int lane = threadIdx.x % kGroup;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup;
    auto fetch = [&](int slot, int64_t r) {
        if (r < rows) {
            R::fetch(ring + slot * kStage, x, r, rows, D, lane);
            R::fetch(ring + slot * kStage + kTensorBytes<T>, dy, r, rows, D, lane);
        }
        copy_commit();
    };
    griddep_wait();
    griddep_launch_dependents();
#pragma unroll
    for (int s = 0; s < kStages - kBatch; ++s) fetch(s, row + s * stride);
    float g[kLnN], dg[kLnN], db[kLnN];
    load_params<R>(gamma, D, lane, 1.0f, g);
#pragma unroll
    for (int i = 0; i < kLnN; ++i) dg[i] = 0.0f, db[i] = 0.0f;
    const float inv_d = 1.0f / static_cast<float>(D);
    // the rows' statistics, loaded a round ahead
    float next_mean[kBatch], next_rstd[kBatch];
    auto load_stats = [&](int64_t first) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool live = first + k * stride < rows;
            next_mean[k] = live ? __ldg(mean_in + first + k * stride) : 0.0f;
            next_rstd[k] = live ? __ldg(rstd_in + first + k * stride) : 0.0f;
        }
    };
    load_stats(row);
    int slot = 0;
    for (; row < rows; row += kBatch * stride) {
        float mean[kBatch], rstd[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) mean[k] = next_mean[k], rstd[k] = next_rstd[k];
        load_stats(row + kBatch * stride);
        copy_wait<kStages - 2 * kBatch>();
        if constexpr (!kAligned) {  // the rows were copied by the whole group
            if constexpr (kGroup > 32) group_barrier(1 + threadIdx.x / kGroup, kGroup);
            else __syncwarp();
        }
        const int last = slot == 0 ? kStages - kBatch : slot - kBatch;  // read in the last round
#pragma unroll
        for (int k = 0; k < kBatch; ++k) fetch(last + k, row + (kStages - kBatch + k) * stride);
        float s[2 * kBatch];  // per row, the sums of g dy and of g dy xhat
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool live = row + k * stride < rows;
            const uint8_t* xs = ring + (slot + k) * kStage;
            const uint8_t* ds = xs + kTensorBytes<T>;
            s[2 * k] = 0.0f;
            s[2 * k + 1] = 0.0f;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                if (live && R::index(i, lane) < D) {
                    const auto px = R::get(xs, x, row + k * stride, D, i, lane);
                    const auto pd = R::get(ds, dy, row + k * stride, D, i, lane);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const int n = i * kVec + e;
                        const float d = to_float(pd.v[e]);
                        const float xhat = (to_float(px.v[e]) - mean[k]) * rstd[k];
                        const float dgx = d * g[n];
                        dg[n] = fmaf(d, xhat, dg[n]);
                        db[n] += d;
                        s[2 * k] += dgx;
                        s[2 * k + 1] = fmaf(dgx, xhat, s[2 * k + 1]);
                    }
                }
            }
        }
        sum(s);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t r = row + k * stride;
            if (r >= rows) break;
            const uint8_t* xs = ring + (slot + k) * kStage;
            const uint8_t* ds = xs + kTensorBytes<T>;
            const float sg = s[2 * k] * inv_d, sgx = s[2 * k + 1] * inv_d;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int j = R::index(i, lane);
                if (j < D) {
                    const auto px = R::get(xs, x, r, D, i, lane);
                    const auto pd = R::get(ds, dy, r, D, i, lane);
                    Pack<T, kVec> p;
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const float xhat = (to_float(px.v[e]) - mean[k]) * rstd[k];
                        const float t = fmaf(to_float(pd.v[e]), g[i * kVec + e], -sg);
                        p.v[e] = from_float<T>(rstd[k] * fmaf(-xhat, sgx, t));
                    }
                    *reinterpret_cast<Pack<T, kVec>*>(dx + r * D + j) = p;
                }
            }
        }
        slot = slot + kBatch == kStages ? 0 : slot + kBatch;
    }
    if (partial == nullptr) return;
    // the block's row of partial sums: its groups own the same columns, and meet in the ring in group order
    float* mine = partial + static_cast<int64_t>(blockIdx.x) * 2 * D;
    copy_wait<0>();
    __syncthreads();
    float* acc = reinterpret_cast<float*>(ring);  // [kRows][2][kGroup * kLnN]
    static_assert(kLnSmemBytes<T, true> >= 2 * kLnThreads * kLnN * 4, "the sums fit the ring");
    constexpr int kCols = kGroup * kLnN;
    float* own = acc + (threadIdx.x / kGroup) * 2 * kCols;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            own[R::index(i, lane) + e] = dg[i * kVec + e];
            own[kCols + R::index(i, lane) + e] = db[i * kVec + e];
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += kLnThreads) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) a += acc[2 * r * kCols + j], b += acc[(2 * r + 1) * kCols + j];
        mine[j] = a;
        mine[D + j] = b;
    }
}

// Long rows: the row's two sums, then dx and the column sums of the block's rows, each pass reading
// x and dy again. A block owns rows b, b + grid, ...; its partial row is summed in global memory by
// the thread that owns the column, in row order.
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    k_ln_bwd_long(const T* dy, const T* x, const Param gamma, const float* __restrict__ mean_in,
                  const float* __restrict__ rstd_in, T* dx, int64_t rows, int32_t D, float* __restrict__ partial) {
    __shared__ float buf[2][2][kLnThreads / 32];
    GroupSum<kLongThreads, 2> sum{buf};
    griddep_wait();
    griddep_launch_dependents();
    const float inv_d = 1.0f / static_cast<float>(D);
    float* mine = partial ? partial + static_cast<int64_t>(blockIdx.x) * 2 * D : nullptr;
    bool first = true;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, first = false) {
        const float mean = mean_in[row], rstd = rstd_in[row];
        const T *xr = x + row * D, *dr = dy + row * D;
        float s[2] = {0.0f, 0.0f};
        for (int j = threadIdx.x; j < D; j += kLongThreads) {
            float g[1];
            load_param<1>(gamma, j, 1.0f, g);
            const float d = to_float(dr[j]), xhat = (to_float(xr[j]) - mean) * rstd;
            s[0] += d * g[0];
            s[1] += d * g[0] * xhat;
        }
        sum(s);
        s[0] *= inv_d;
        s[1] *= inv_d;
        for (int j = threadIdx.x; j < D; j += kLongThreads) {
            float g[1];
            load_param<1>(gamma, j, 1.0f, g);
            const float d = to_float(dr[j]), xhat = (to_float(xr[j]) - mean) * rstd;
            dx[row * D + j] = from_float<T>(rstd * (d * g[0] - s[0] - xhat * s[1]));
            if (mine) {
                mine[j] = (first ? 0.0f : mine[j]) + d * xhat;
                mine[D + j] = (first ? 0.0f : mine[D + j]) + d;
            }
        }
    }
}

// dgamma[j] = sum over the blocks' partial rows in block order; dbeta likewise. A block owns 32
// columns of one of the two sums; its warps take the rows in turn and meet in shared memory.
constexpr int kGradWarps = 16;
__global__ void __launch_bounds__(32 * kGradWarps)
    k_ln_param_grads(const float* __restrict__ partial, int32_t blocks, int32_t D, int32_t param_dtype,
                     void* __restrict__ dgamma, void* __restrict__ dbeta) {
    __shared__ float acc[kGradWarps][32];
    griddep_wait();
    griddep_launch_dependents();
    void* out = blockIdx.y == 0 ? dgamma : dbeta;
    if (out == nullptr) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + lane;
    // all of a warp's rows at once: one latency instead of one per row
    float v[(kLnMaxBlocks + kGradWarps - 1) / kGradWarps];
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < static_cast<int>(sizeof(v) / sizeof(v[0])); ++u) {
        const int b = warp + u * kGradWarps;
        v[u] = j < D && b < blocks ? partial[(static_cast<int64_t>(b) * 2 + blockIdx.y) * D + j] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < static_cast<int>(sizeof(v) / sizeof(v[0])); ++u) s += v[u];
    acc[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && j < D) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradWarps; ++w) s += acc[w][lane];
        store_param(out, param_dtype, j, s);
    }
}

// One block per SM, fewer for few rows.
int ln_grid(const LayerNormProblem& p, int rows_per_block) {
    return static_cast<int>(std::min<int64_t>(
        {ceil_div(p.T, rows_per_block), static_cast<int64_t>(p.sm_count), static_cast<int64_t>(kLnMaxBlocks)}));
}

template <typename T, int kGroup, bool kAligned>
cudaError_t run_fwd(const LayerNormProblem& p, cudaStream_t stream) {
    constexpr int kBytes = kLnSmemBytes<T, false>;
    const cudaError_t e = allow_smem<&k_ln_fwd<T, kGroup, kAligned>>(kBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_ln_fwd<T, kGroup, kAligned>, dim3(ln_grid(p, kLnThreads / kGroup)),
                      dim3(kLnThreads), kBytes, stream, static_cast<const T*>(p.x), param(p.gamma, p.param_dtype),
                      param(p.beta, p.param_dtype), static_cast<T*>(p.y), p.mean, p.rstd, p.T, p.D, p.eps);
}

template <typename T, bool kAligned>
cudaError_t dispatch_fwd(const LayerNormProblem& p, cudaStream_t stream) {
    if (p.D <= 512) return run_fwd<T, 32, kAligned>(p, stream);
    if (p.D <= 1024) return run_fwd<T, 64, kAligned>(p, stream);
    if (p.D <= 2048) return run_fwd<T, 128, kAligned>(p, stream);
    if (p.D <= 4096) return run_fwd<T, 256, kAligned>(p, stream);
    return run_fwd<T, 512, kAligned>(p, stream);
}

template <typename T>
cudaError_t fwd_of(const LayerNormProblem& p, cudaStream_t stream) {
    if (p.D > kLnThreads * kLnN)
        return launch_pdl(k_ln_fwd_long<T>, dim3(static_cast<unsigned>(p.T)), dim3(kLongThreads), 0, stream,
                          static_cast<const T*>(p.x), param(p.gamma, p.param_dtype), param(p.beta, p.param_dtype),
                          static_cast<T*>(p.y), p.mean, p.rstd, p.D, p.eps);
    const int64_t bytes = static_cast<int64_t>(p.D) * sizeof(T);
    return rows_aligned16(p.x, bytes) && rows_aligned16(p.y, bytes) ? dispatch_fwd<T, true>(p, stream)
                                                                   : dispatch_fwd<T, false>(p, stream);
}

template <typename T, int kGroup, bool kAligned>
cudaError_t run_bwd(const LayerNormProblem& p, int* blocks, cudaStream_t stream) {
    constexpr int kBytes = kLnSmemBytes<T, true>;
    const cudaError_t e = allow_smem<&k_ln_bwd<T, kGroup, kAligned>>(kBytes);
    if (e != cudaSuccess) return e;
    *blocks = ln_grid(p, kLnThreads / kGroup);
    return launch_pdl(k_ln_bwd<T, kGroup, kAligned>, dim3(*blocks), dim3(kLnThreads), kBytes, stream,
                      static_cast<const T*>(p.dy), static_cast<const T*>(p.x), param(p.gamma, p.param_dtype), p.mean_in,
                      p.rstd_in, static_cast<T*>(p.dx), p.T, p.D, p.partial);
}

template <typename T, bool kAligned>
cudaError_t dispatch_bwd(const LayerNormProblem& p, int* blocks, cudaStream_t stream) {
    if (p.D <= 512) return run_bwd<T, 32, kAligned>(p, blocks, stream);
    if (p.D <= 1024) return run_bwd<T, 64, kAligned>(p, blocks, stream);
    if (p.D <= 2048) return run_bwd<T, 128, kAligned>(p, blocks, stream);
    if (p.D <= 4096) return run_bwd<T, 256, kAligned>(p, blocks, stream);
    return run_bwd<T, 512, kAligned>(p, blocks, stream);
}

template <typename T>
cudaError_t bwd_of(const LayerNormProblem& p, int* blocks, cudaStream_t stream) {
    if (p.D > kLnThreads * kLnN) {
        *blocks = ln_grid(p, 1);
        return launch_pdl(k_ln_bwd_long<T>, dim3(*blocks), dim3(kLongThreads), 0, stream, static_cast<const T*>(p.dy),
                          static_cast<const T*>(p.x), param(p.gamma, p.param_dtype), p.mean_in, p.rstd_in,
                          static_cast<T*>(p.dx), p.T, p.D, p.partial);
    }
    const int64_t bytes = static_cast<int64_t>(p.D) * sizeof(T);
    return rows_aligned16(p.x, bytes) && rows_aligned16(p.dy, bytes) && rows_aligned16(p.dx, bytes)
               ? dispatch_bwd<T, true>(p, blocks, stream)
               : dispatch_bwd<T, false>(p, blocks, stream);
}

}  // namespace

moe_status_t launch_layernorm_fwd(const LayerNormProblem& p, cudaStream_t stream) {
    const cudaError_t e = p.dtype == MOE_DTYPE_F32    ? fwd_of<float>(p, stream)
                          : p.dtype == MOE_DTYPE_BF16 ? fwd_of<__nv_bfloat16>(p, stream)
                                                      : fwd_of<__half>(p, stream);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t launch_layernorm_bwd(const LayerNormProblem& in, cudaStream_t stream) {
    LayerNormProblem p = in;
    if (!p.dgamma && !p.dbeta) p.partial = nullptr;
    int blocks = 0;
    cudaError_t e = p.dtype == MOE_DTYPE_F32    ? bwd_of<float>(p, &blocks, stream)
                    : p.dtype == MOE_DTYPE_BF16 ? bwd_of<__nv_bfloat16>(p, &blocks, stream)
                                                : bwd_of<__half>(p, &blocks, stream);
    if (e == cudaSuccess && p.partial)
        e = launch_pdl(k_ln_param_grads, dim3(static_cast<unsigned>(ceil_div(p.D, 32)), 2), dim3(32 * kGradWarps), 0,
                       stream, static_cast<const float*>(p.partial), static_cast<int32_t>(blocks), p.D, p.param_dtype,
                       p.dgamma, p.dbeta);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
