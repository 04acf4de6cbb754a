// router.cu -- the top-k router: expert ids and scores from router logits, and the way back from
// the scores' gradient to the logits'.
//
//   ids[t, :] = the K largest of z[t, :], largest first, equal logits by the lowest expert id
//   normalize:  scores = softmax of the K chosen logits
//   otherwise:  scores = the softmax over all E experts, at the chosen ones
//   backward:   normalize:  dz_i = s_i (ds_i - sum_j s_j ds_j) at the chosen experts, 0 elsewhere
//               otherwise:  dz_i = p_i ([i chosen] ds_i - sum_j s_j ds_j) at every expert
//
// A logit of -inf masks its expert: its probability is 0, and it is chosen only when fewer than K
// experts are left. A row with nothing but -inf gets scores of 0 and a gradient of 0. A NaN sorts
// above everything, as a failure that has to show: the row's scores are NaN.
//
// Both directions read or write T E logits once and are bound by that traffic. One warp owns a
// row (up to 1024 experts; 4 warps up to 4096) and holds it in registers as order-preserving
// integer keys, so that each of the K rounds is a maximum over the lane's keys, one warp-wide
// maximum of the key and one warp-wide minimum of the index.
#include "ptx_sm103.cuh"
#include "train_internal.cuh"

namespace moe {
namespace {

constexpr int kRouterThreads = 128;

// The float's position in the order of the reals as an unsigned integer; never 0. -0 equals +0,
// every NaN is the largest.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0xffffffffu;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// Element i of a thread's kN: kVec consecutive experts at a time, kThreads threads side by side.
// Ascending in i, so the first of a thread's equal keys is the one with the lowest expert id.
template <int kThreads, int kVec>
__device__ __forceinline__ int expert_of(int i, int t) {
    return (i / kVec) * kThreads * kVec + t * kVec + i % kVec;
}

template <typename T, int kVec>
struct alignas(sizeof(T) * kVec) LogitPack {
    T v[kVec];
};

// Reductions over the kThreads threads of a row: one warp, or the block through shared memory with
// alternating buffers (a buffer is written again only after the next reduction's barrier).
template <int kThreads>
struct RowReduce {
    uint2 (*buf)[kThreads / 32];
    int turn = 0;
    __device__ uint2 argmax(uint32_t key, int idx) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, key);
        uint2 r = make_uint2(best, __reduce_min_sync(0xffffffffu, key == best ? static_cast<uint32_t>(idx) : 0xffffffffu));
        if constexpr (kThreads > 32) {
            uint2* b = buf[turn];
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = r;
            __syncthreads();
            r = b[0];
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w)
                if (b[w].x > r.x || (b[w].x == r.x && b[w].y < r.y)) r = b[w];
        }
        return r;
    }
    __device__ float sum(float v) {
        v = warp_sum(v);
        if constexpr (kThreads > 32) {
            uint2* b = buf[turn];
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = make_uint2(__float_as_uint(v), 0u);
            __syncthreads();
            v = 0.0f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) v += __uint_as_float(b[w].x);
        }
        return v;
    }
};

template <typename T, int kThreads, int kN, int kVec>
__global__ void __launch_bounds__(kRouterThreads)
    k_router_fwd(const T* __restrict__ logits, int64_t rows, int32_t E, int32_t K, bool normalize,
                 int32_t* __restrict__ ids, float* __restrict__ scores) {
    __shared__ uint2 buf[2][kThreads / 32];
    RowReduce<kThreads> red{buf};
    const int t = threadIdx.x % kThreads;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRouterThreads / kThreads) + threadIdx.x / kThreads;
    griddep_wait();
    griddep_launch_dependents();
    if (row >= rows) return;  // whole warps, or (one row per block) never
    uint32_t key[kN];
#pragma unroll
    for (int i = 0; i < kN; i += kVec) {
        const int e0 = expert_of<kThreads, kVec>(i, t);
        if (e0 < E) {
            const auto p = *reinterpret_cast<const LogitPack<T, kVec>*>(logits + row * E + e0);
#pragma unroll
            for (int e = 0; e < kVec; ++e) key[i + e] = order_key(to_float(p.v[e]));
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) key[i + e] = 0u;
        }
    }
    float m = 0.0f, total = 0.0f;
    int32_t* my_ids = ids + row * K;
    float* my_scores = scores + row * K;
    int32_t id_k = 0;  // lane k % 32 keeps choice k until 32 of them are stored at once
    float v_k = 0.0f, e_k = 0.0f, part = 0.0f;
    for (int k = 0; k < K; ++k) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint2 top = red.argmax(best, expert_of<kThreads, kVec>(at, t));
        if (k == 0) {
            m = key_value(top.x);
            if (!normalize) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < kN; ++i)
                    if (key[i] != 0u) s += expf(key_value(key[i]) - m);
                total = red.sum(s);
            }
        }
        if (t == (k & 31)) {
            id_k = static_cast<int32_t>(top.y);
            v_k = key_value(top.x);
        }
        const int own = static_cast<int>(top.y) - t * kVec;  // its place among this thread's, if it is one
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (own == expert_of<kThreads, kVec>(i, 0)) key[i] = 0u;
        if ((k & 31) == 31 && t < 32) {  // a warp's worth of choices; scaled below
            e_k = expf(v_k - m);
            part += e_k;
            my_ids[k - 31 + t] = id_k;
            my_scores[k - 31 + t] = e_k;
        }
    }
    if (t >= 32) return;
    const int rest = K & ~31;  // choices [rest, K) are still in registers
    const bool mine = rest + t < K;
    if (mine) {
        e_k = expf(v_k - m);
        part += e_k;
    }
    if (normalize) total = warp_sum(part);
    const bool none = m == -INFINITY;  // a row with nothing but -inf has scores of 0
    const float inv = 1.0f / total;
    if (mine) {
        my_ids[rest + t] = id_k;
        my_scores[rest + t] = none ? 0.0f : e_k * inv;
    }
    for (int k = t; k < rest; k += 32) my_scores[k] = none ? 0.0f : my_scores[k] * inv;  // as this thread wrote it
}

template <typename T, int kThreads, int kN, int kVec>
__global__ void __launch_bounds__(kRouterThreads)
    k_router_bwd(const T* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ dscores,
                 int64_t rows, int32_t E, int32_t K, bool normalize, T* __restrict__ dlogits) {
    __shared__ uint2 buf[2][kThreads / 32];
    RowReduce<kThreads> red{buf};
    const int t = threadIdx.x % kThreads;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRouterThreads / kThreads) + threadIdx.x / kThreads;
    griddep_wait();
    griddep_launch_dependents();
    if (row >= rows) return;
    // the scores' gradients at this thread's experts; an id outside [0, E) matches none of them
    float ds[kN];
    bool chosen[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) ds[i] = 0.0f, chosen[i] = false;
    for (int k = 0; k < K; ++k) {
        const int32_t id = __ldg(ids + row * K + k);
        const float d = __ldg(dscores + row * K + k);
        const bool inside = id >= 0 && id < E;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (inside && expert_of<kThreads, kVec>(i, t) == id) ds[i] += d, chosen[i] = true;
    }
    float z[kN];
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < kN; i += kVec) {
        const int e0 = expert_of<kThreads, kVec>(i, t);
        bool need = !normalize;
#pragma unroll
        for (int e = 0; e < kVec; ++e) need = need || chosen[i + e];
        if (e0 < E && need) {
            const auto p = *reinterpret_cast<const LogitPack<T, kVec>*>(logits + row * E + e0);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const bool in = !normalize || chosen[i + e];
                z[i + e] = in ? to_float(p.v[e]) : -INFINITY;
                if (in) best = max(best, order_key(z[i + e]));
            }
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) z[i + e] = -INFINITY;
        }
    }
    const uint32_t top = red.argmax(best, t).x;
    const float m = top == 0u ? -INFINITY : key_value(top);
    const bool none = m == -INFINITY;  // nothing chosen, or everything masked: no gradient
    float s = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        z[i] = none ? 0.0f : expf(z[i] - m);
        s += z[i];
    }
    s = red.sum(s);
    const float inv = none ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        z[i] *= inv;
        dot += chosen[i] ? z[i] * ds[i] : 0.0f;
    }
    dot = red.sum(dot);
#pragma unroll
    for (int i = 0; i < kN; i += kVec) {
        const int e0 = expert_of<kThreads, kVec>(i, t);
        if (e0 < E) {
            LogitPack<T, kVec> p;
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                p.v[e] = from_float<T>(none || (normalize && !chosen[i + e]) ? 0.0f : z[i + e] * (ds[i + e] - dot));
            *reinterpret_cast<LogitPack<T, kVec>*>(dlogits + row * E + e0) = p;
        }
    }
}

template <typename T, int kThreads, int kN, int kVec>
cudaError_t run(const RouterProblem& p, bool fwd, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(ceil_div(p.T, kRouterThreads / kThreads)));
    if (fwd)
        return launch_pdl(k_router_fwd<T, kThreads, kN, kVec>, grid, dim3(kRouterThreads), 0, stream,
                          static_cast<const T*>(p.logits), p.T, p.E, p.K, p.normalize, p.ids, p.scores);
    return launch_pdl(k_router_bwd<T, kThreads, kN, kVec>, grid, dim3(kRouterThreads), 0, stream,
                      static_cast<const T*>(p.logits), p.ids_in, p.dscores, p.T, p.E, p.K, p.normalize,
                      static_cast<T*>(p.dlogits));
}

template <typename T, int kVec>
cudaError_t dispatch(const RouterProblem& p, bool fwd, cudaStream_t stream) {
    if (p.E <= 128) return run<T, 32, 4, kVec>(p, fwd, stream);
    if (p.E <= 256) return run<T, 32, 8, kVec>(p, fwd, stream);
    if (p.E <= 512) return run<T, 32, 16, kVec>(p, fwd, stream);
    if (p.E <= 1024) return run<T, 32, 32, kVec>(p, fwd, stream);
    return run<T, 128, 32, kVec>(p, fwd, stream);
}

// Four experts per load where every row starts on such a boundary, one otherwise.
template <typename T>
moe_status_t launch(const RouterProblem& p, bool fwd, cudaStream_t stream) {
    const size_t pack = 4 * sizeof(T);
    const bool vec = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % pack == 0 &&
                     (fwd || reinterpret_cast<uintptr_t>(p.dlogits) % pack == 0);
    return (vec ? dispatch<T, 4>(p, fwd, stream) : dispatch<T, 1>(p, fwd, stream)) == cudaSuccess ? MOE_OK
                                                                                                 : MOE_ERR_CUDA;
}

}  // namespace

moe_status_t launch_router_fwd(const RouterProblem& p, cudaStream_t stream) {
    return p.dtype == MOE_DTYPE_F32 ? launch<float>(p, true, stream) : launch<__nv_bfloat16>(p, true, stream);
}

moe_status_t launch_router_bwd(const RouterProblem& p, cudaStream_t stream) {
    return p.dtype == MOE_DTYPE_F32 ? launch<float>(p, false, stream) : launch<__nv_bfloat16>(p, false, stream);
}

}  // namespace moe
