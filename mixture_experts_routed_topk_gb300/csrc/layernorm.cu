// layernorm.cu -- layer norm over the last dimension, forward and backward.
//
//   mean = sum_d x / D,  rstd = 1 / sqrt(sum_d (x - mean)^2 / D + eps),  xhat = (x - mean) rstd
//   y = xhat gamma + beta
//   with g = dy gamma:  dx = rstd (g - mean_d(g) - xhat mean_d(g xhat))
//   dgamma = sum_t dy xhat,  dbeta = sum_t dy
//
// Both directions are bound by memory: forward T D read and written once, backward 2 T D read and
// T D written. A row is read once and stays in registers (rows up to 8192 elements; longer ones
// are read again, mostly from L2). All arithmetic is fp32; the variance is taken from the centred
// values, so a large mean does not cancel it away.
//
// The backward grid is persistent: a block walks rows b, b + grid, ... and keeps its column sums of
// dy xhat and dy in registers, so dgamma and dbeta cost no extra pass over x and dy. Each block
// writes one row of partial sums, and a second kernel adds the rows in block order: the result
// does not depend on the order in which blocks finish.
#include <algorithm>

#include "ptx_sm103.cuh"
#include "train_internal.cuh"

namespace moe {
namespace {

// One thread's piece of a row: kN / kVec vectors of kVec elements, vector i at element
// (i * kGroup + lane) * kVec of the row. kVec elements fill 16 bytes, or kVec is 1 where the rows
// do not all start on 16-byte boundaries.
template <typename T, int kVec>
struct alignas(sizeof(T) * kVec) Pack {
    T v[kVec];
};

// gamma or beta: their type and whether 16-byte loads of them are aligned, or null.
struct Param {
    const void* p;
    int32_t dtype;
    bool vec;
};

template <typename P, int kVec>
__device__ __forceinline__ void load_param_as(const void* base, bool vec, int j, float (&out)[kVec]) {
    const P* p = static_cast<const P*>(base) + j;
    if (kVec > 1 && vec) {
        constexpr int kStep = kVec > 1 ? (16 / sizeof(P) < kVec ? 16 / sizeof(P) : kVec) : 1;
#pragma unroll
        for (int e = 0; e < kVec; e += kStep) {
            const auto q = *reinterpret_cast<const Pack<P, kStep>*>(p + e);
#pragma unroll
            for (int i = 0; i < kStep; ++i) out[e + i] = to_float(q.v[i]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) out[e] = to_float(p[e]);
    }
}

template <int kVec>
__device__ __forceinline__ void load_param(const Param& a, int j, float none, float (&out)[kVec]) {
    if (a.p == nullptr) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) out[e] = none;
    } else if (a.dtype == MOE_DTYPE_F32) {
        load_param_as<float, kVec>(a.p, a.vec, j, out);
    } else if (a.dtype == MOE_DTYPE_BF16) {
        load_param_as<__nv_bfloat16, kVec>(a.p, a.vec, j, out);
    } else {
        load_param_as<__half, kVec>(a.p, a.vec, j, out);
    }
}

__device__ __forceinline__ void store_param(void* p, int32_t dtype, int64_t j, float v) {
    if (dtype == MOE_DTYPE_F32) static_cast<float*>(p)[j] = v;
    else if (dtype == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(p)[j] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[j] = __float2half_rn(v);
}

// Sum over the kGroup threads of a row; every thread of the group gets it. kGroup is 32 (one warp)
// or the whole block. The two buffers alternate, so that one barrier per sum is enough: a warp
// writes buffer b again only after the barrier of the sum in between, which every reader has passed.
template <int kGroup>
struct GroupSum {
    float (*buf)[32];
    int turn = 0;
    __device__ float operator()(float v) {
        v = warp_sum(v);
        if constexpr (kGroup > 32) {
            float* b = buf[turn];
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
            __syncthreads();
            v = 0.0f;
#pragma unroll
            for (int w = 0; w < kGroup / 32; ++w) v += b[w];
        }
        return v;
    }
};

constexpr int kWarpBlock = 128;  // threads of a block whose warps own a row each
template <int kGroup>
constexpr int kBlockThreads = kGroup == 32 ? kWarpBlock : kGroup;

// x and y are not declared restrict: y may be x itself (a row is in registers before it is written).
template <typename T, int kGroup, int kN, int kVec>
__global__ void __launch_bounds__(kBlockThreads<kGroup>)
    k_ln_fwd(const T* x, const Param gamma, const Param beta, T* y, float* __restrict__ mean_out,
             float* __restrict__ rstd_out, int64_t rows, int32_t D, float eps) {
    constexpr int kRows = kBlockThreads<kGroup> / kGroup;
    constexpr int kVecs = kN / kVec;
    using P = Pack<T, kVec>;
    __shared__ float buf[2][32];
    GroupSum<kGroup> sum{buf};
    const int lane = threadIdx.x % kGroup;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup;
    griddep_wait();
    griddep_launch_dependents();
    if (row >= rows) return;  // whole warps; a block that is one group always has its row
    const T* xr = x + row * D;
    float v[kN];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int j = (i * kGroup + lane) * kVec;
        if (j < D) {
            const P p = *reinterpret_cast<const P*>(xr + j);
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[i * kVec + e] = to_float(p.v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[i * kVec + e] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) s += v[i];
    const float inv_d = 1.0f / static_cast<float>(D);
    const float mean = sum(s) * inv_d;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        if ((i * kGroup + lane) * kVec < D) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float c = v[i * kVec + e] - mean;
                v[i * kVec + e] = c;
                q += c * c;
            }
        }
    }
    const float rstd = 1.0f / sqrtf(sum(q) * inv_d + eps);
    T* yr = y + row * D;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int j = (i * kGroup + lane) * kVec;
        if (j < D) {
            float g[kVec], b[kVec];
            load_param<kVec>(gamma, j, 1.0f, g);
            load_param<kVec>(beta, j, 0.0f, b);
            P p;
#pragma unroll
            for (int e = 0; e < kVec; ++e) p.v[e] = from_float<T>(fmaf(v[i * kVec + e] * rstd, g[e], b[e]));
            *reinterpret_cast<P*>(yr + j) = p;
        }
    }
    if (lane == 0) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }
}

// Rows longer than the registers hold: three passes over the row, the second and third from L2.
constexpr int kLongThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    k_ln_fwd_long(const T* x, const Param gamma, const Param beta, T* y, float* __restrict__ mean_out,
                  float* __restrict__ rstd_out, int32_t D, float eps) {
    __shared__ float buf[2][32];
    GroupSum<kLongThreads> sum{buf};
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* xr = x + row * D;
    const float inv_d = 1.0f / static_cast<float>(D);
    float s = 0.0f;
    for (int j = threadIdx.x; j < D; j += kLongThreads) s += to_float(xr[j]);
    const float mean = sum(s) * inv_d;
    float q = 0.0f;
    for (int j = threadIdx.x; j < D; j += kLongThreads) {
        const float c = to_float(xr[j]) - mean;
        q += c * c;
    }
    const float rstd = 1.0f / sqrtf(sum(q) * inv_d + eps);
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
template <typename T, int kGroup, int kN, int kVec>
__global__ void __launch_bounds__(kBlockThreads<kGroup>)
    k_ln_bwd(const T* dy, const T* x, const Param gamma, const float* __restrict__ mean_in,
             const float* __restrict__ rstd_in, T* dx, int64_t rows, int32_t D, float* __restrict__ partial) {
    constexpr int kRows = kBlockThreads<kGroup> / kGroup;
    constexpr int kVecs = kN / kVec;
    using P = Pack<T, kVec>;
    __shared__ float buf[2][32];
    GroupSum<kGroup> sum{buf};
    const int lane = threadIdx.x % kGroup;
    float dg[kN], db[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) dg[i] = 0.0f, db[i] = 0.0f;
    griddep_wait();
    griddep_launch_dependents();
    const float inv_d = 1.0f / static_cast<float>(D);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup; row < rows;
         row += static_cast<int64_t>(gridDim.x) * kRows) {
        P px[kVecs], pd[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = (i * kGroup + lane) * kVec;
            if (j < D) {
                px[i] = *reinterpret_cast<const P*>(x + row * D + j);
                pd[i] = *reinterpret_cast<const P*>(dy + row * D + j);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) px[i].v[e] = from_float<T>(0.0f), pd[i].v[e] = from_float<T>(0.0f);
            }
        }
        const float mean = mean_in[row], rstd = rstd_in[row];
        float sg = 0.0f, sgx = 0.0f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = (i * kGroup + lane) * kVec;
            if (j < D) {
                float g[kVec];
                load_param<kVec>(gamma, j, 1.0f, g);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float d = to_float(pd[i].v[e]);
                    const float xhat = (to_float(px[i].v[e]) - mean) * rstd;
                    dg[i * kVec + e] += d * xhat;
                    db[i * kVec + e] += d;
                    sg += d * g[e];
                    sgx += d * g[e] * xhat;
                }
            }
        }
        sg = sum(sg) * inv_d;
        sgx = sum(sgx) * inv_d;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = (i * kGroup + lane) * kVec;
            if (j < D) {
                float g[kVec];
                load_param<kVec>(gamma, j, 1.0f, g);
                P p;
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float xhat = (to_float(px[i].v[e]) - mean) * rstd;
                    p.v[e] = from_float<T>(rstd * (to_float(pd[i].v[e]) * g[e] - sg - xhat * sgx));
                }
                *reinterpret_cast<P*>(dx + row * D + j) = p;
            }
        }
    }
    if (partial == nullptr) return;
    float* mine = partial + static_cast<int64_t>(blockIdx.x) * 2 * D;
    if constexpr (kRows > 1) {
        // the block's warps own the same columns: add them in warp order
        __shared__ float acc[2][kGroup * kN];
        for (int w = 0; w < kRows; ++w) {
            __syncthreads();
            if (static_cast<int>(threadIdx.x) / kGroup == w) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const int j = (i * kGroup + lane) * kVec + e;
                        acc[0][j] = (w ? acc[0][j] : 0.0f) + dg[i * kVec + e];
                        acc[1][j] = (w ? acc[1][j] : 0.0f) + db[i * kVec + e];
                    }
                }
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < D; j += blockDim.x) {
            mine[j] = acc[0][j];
            mine[D + j] = acc[1][j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const int j = (i * kGroup + lane) * kVec + e;
                if (j < D) {
                    mine[j] = dg[i * kVec + e];
                    mine[D + j] = db[i * kVec + e];
                }
            }
        }
    }
}

// Long rows: the row's two sums, then dx and the column sums of the block's rows, each pass reading
// x and dy again. A block owns rows b, b + grid, ...; its partial row is summed in global memory by
// the thread that owns the column, in row order.
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    k_ln_bwd_long(const T* dy, const T* x, const Param gamma, const float* __restrict__ mean_in,
                  const float* __restrict__ rstd_in, T* dx, int64_t rows, int32_t D, float* __restrict__ partial) {
    __shared__ float buf[2][32];
    GroupSum<kLongThreads> sum{buf};
    griddep_wait();
    griddep_launch_dependents();
    const float inv_d = 1.0f / static_cast<float>(D);
    float* mine = partial ? partial + static_cast<int64_t>(blockIdx.x) * 2 * D : nullptr;
    bool first = true;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, first = false) {
        const float mean = mean_in[row], rstd = rstd_in[row];
        const T *xr = x + row * D, *dr = dy + row * D;
        float sg = 0.0f, sgx = 0.0f;
        for (int j = threadIdx.x; j < D; j += kLongThreads) {
            float g[1];
            load_param<1>(gamma, j, 1.0f, g);
            const float d = to_float(dr[j]), xhat = (to_float(xr[j]) - mean) * rstd;
            sg += d * g[0];
            sgx += d * g[0] * xhat;
        }
        sg = sum(sg) * inv_d;
        sgx = sum(sgx) * inv_d;
        for (int j = threadIdx.x; j < D; j += kLongThreads) {
            float g[1];
            load_param<1>(gamma, j, 1.0f, g);
            const float d = to_float(dr[j]), xhat = (to_float(xr[j]) - mean) * rstd;
            dx[row * D + j] = from_float<T>(rstd * (d * g[0] - sg - xhat * sgx));
            if (mine) {
                mine[j] = (first ? 0.0f : mine[j]) + d * xhat;
                mine[D + j] = (first ? 0.0f : mine[D + j]) + d;
            }
        }
    }
}

// dgamma[j] = sum over the blocks' partial rows in block order; dbeta likewise. A block owns 32
// columns of one of the two sums; its warps take the rows in turn and meet in shared memory.
constexpr int kGradWarps = 8;
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
    float s = 0.0f;
    if (j < D)
        for (int b = warp; b < blocks; b += kGradWarps)
            s += partial[(static_cast<int64_t>(b) * 2 + blockIdx.y) * D + j];
    acc[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && j < D) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradWarps; ++w) s += acc[w][lane];
        store_param(out, param_dtype, j, s);
    }
}

bool rows_aligned16(const void* p, int64_t row_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0;
}

Param param(const void* p, int32_t dtype) { return Param{p, dtype, reinterpret_cast<uintptr_t>(p) % 16 == 0}; }

template <typename T, int kGroup, int kN, int kVec>
cudaError_t run_fwd(const LayerNormProblem& p, cudaStream_t stream) {
    constexpr int kRows = kBlockThreads<kGroup> / kGroup;
    return launch_pdl(k_ln_fwd<T, kGroup, kN, kVec>, dim3(static_cast<unsigned>(ceil_div(p.T, kRows))),
                      dim3(kBlockThreads<kGroup>), 0, stream, static_cast<const T*>(p.x),
                      param(p.gamma, p.param_dtype), param(p.beta, p.param_dtype), static_cast<T*>(p.y), p.mean, p.rstd,
                      p.T, p.D, p.eps);
}

template <typename T, int kVec>
cudaError_t dispatch_fwd(const LayerNormProblem& p, cudaStream_t stream) {
    if (p.D <= 256) return run_fwd<T, 32, 8, kVec>(p, stream);
    if (p.D <= 512) return run_fwd<T, 32, 16, kVec>(p, stream);
    if (p.D <= 1024) return run_fwd<T, 32, 32, kVec>(p, stream);
    if (p.D <= 2048) return run_fwd<T, 128, 16, kVec>(p, stream);
    if (p.D <= 4096) return run_fwd<T, 256, 16, kVec>(p, stream);
    if (p.D <= 8192) return run_fwd<T, 512, 16, kVec>(p, stream);
    return launch_pdl(k_ln_fwd_long<T>, dim3(static_cast<unsigned>(p.T)), dim3(kLongThreads), 0, stream,
                      static_cast<const T*>(p.x), param(p.gamma, p.param_dtype), param(p.beta, p.param_dtype),
                      static_cast<T*>(p.y), p.mean, p.rstd, p.D, p.eps);
}

template <typename T>
cudaError_t fwd_of(const LayerNormProblem& p, cudaStream_t stream) {
    constexpr int kVec = 16 / sizeof(T);
    const int64_t bytes = static_cast<int64_t>(p.D) * sizeof(T);
    return rows_aligned16(p.x, bytes) && rows_aligned16(p.y, bytes) ? dispatch_fwd<T, kVec>(p, stream)
                                                                   : dispatch_fwd<T, 1>(p, stream);
}

int bwd_grid(const LayerNormProblem& p, int rows_per_block, int threads) {
    const int64_t want = ceil_div(p.T, rows_per_block);
    const int64_t per_sm = threads <= 256 ? 2 : 1;
    return static_cast<int>(std::min<int64_t>({want, per_sm * p.sm_count, static_cast<int64_t>(kLnMaxBlocks)}));
}

template <typename T, int kGroup, int kN, int kVec>
cudaError_t run_bwd(const LayerNormProblem& p, int* blocks, cudaStream_t stream) {
    *blocks = bwd_grid(p, kBlockThreads<kGroup> / kGroup, kBlockThreads<kGroup>);
    return launch_pdl(k_ln_bwd<T, kGroup, kN, kVec>, dim3(*blocks), dim3(kBlockThreads<kGroup>), 0, stream,
                      static_cast<const T*>(p.dy), static_cast<const T*>(p.x), param(p.gamma, p.param_dtype), p.mean_in,
                      p.rstd_in, static_cast<T*>(p.dx), p.T, p.D, p.partial);
}

template <typename T, int kVec>
cudaError_t dispatch_bwd(const LayerNormProblem& p, int* blocks, cudaStream_t stream) {
    if (p.D <= 256) return run_bwd<T, 32, 8, kVec>(p, blocks, stream);
    if (p.D <= 512) return run_bwd<T, 32, 16, kVec>(p, blocks, stream);
    if (p.D <= 2048) return run_bwd<T, 128, 16, kVec>(p, blocks, stream);
    if (p.D <= 4096) return run_bwd<T, 256, 16, kVec>(p, blocks, stream);
    if (p.D <= 8192) return run_bwd<T, 512, 16, kVec>(p, blocks, stream);
    *blocks = bwd_grid(p, 1, kLongThreads);
    return launch_pdl(k_ln_bwd_long<T>, dim3(*blocks), dim3(kLongThreads), 0, stream, static_cast<const T*>(p.dy),
                      static_cast<const T*>(p.x), param(p.gamma, p.param_dtype), p.mean_in, p.rstd_in,
                      static_cast<T*>(p.dx), p.T, p.D, p.partial);
}

template <typename T>
cudaError_t bwd_of(const LayerNormProblem& p, int* blocks, cudaStream_t stream) {
    constexpr int kVec = 16 / sizeof(T);
    const int64_t bytes = static_cast<int64_t>(p.D) * sizeof(T);
    return rows_aligned16(p.x, bytes) && rows_aligned16(p.dy, bytes) && rows_aligned16(p.dx, bytes)
               ? dispatch_bwd<T, kVec>(p, blocks, stream)
               : dispatch_bwd<T, 1>(p, blocks, stream);
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
