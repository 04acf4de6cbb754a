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
// Both directions read or write T E logits once. One warp owns a row (up to 1024 experts; 4 warps up to
// 4096) and holds it in registers. The forward's K rounds of selection cost more than that traffic, so:
// where a logit and its expert id fit one 32-bit key without a doubt (bf16 logits; fp32 ones up to 256
// experts by their upper 24 bits, when the first K + 1 of those all differ), each lane sorts its keys once,
// and a round is one warp-wide maximum over the lanes' first keys. Otherwise a round is a search
// through the lane's keys, a warp-wide maximum of the logit and a warp-wide minimum of the id.
// The backward gives each choice a lane; the other experts' gradients need no search.
// 16384 x 256 fp32, K = 8, scores over the chosen: forward 15.1 us with the second kind of round for every row,
// 9.1 us with the first; backward 12.4 us with a search for each choice, 6.6 us without. Scores over all
// experts: forward 11.2 us, backward 7.8 us. bf16: forward 8.3 and 10.2 us. 384 experts, which fp32 keys of 8 id
// bits cannot hold: fp32 23.4 us, bf16 15.8 us.
#include "ptx_sm103.cuh"
#include "train_internal.cuh"

namespace moe {
namespace {

constexpr int kRouterThreads = 128;

// The float's position in the order of the reals as an unsigned integer; never 0. The addition makes
// -0 equal to +0 and every NaN the canonical one, whose key is the largest.
__device__ __forceinline__ uint32_t order_key(float v) {
    const int32_t b = __float_as_int(v + 0.0f);
    return static_cast<uint32_t>(b ^ ((b >> 31) | INT32_MIN));
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

// The keys of this thread's experts; 0 for experts that do not exist.
template <typename T, int kThreads, int kN, int kVec>
__device__ __forceinline__ void load_keys(const T* row, int32_t E, int t, uint32_t (&key)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; i += kVec) {
        const int e0 = expert_of<kThreads, kVec>(i, t);
        if (e0 < E) {
            const auto p = *reinterpret_cast<const LogitPack<T, kVec>*>(row + e0);
#pragma unroll
            for (int e = 0; e < kVec; ++e) key[i + e] = order_key(to_float(p.v[e]));
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) key[i + e] = 0u;
        }
    }
}

// Bits of the expert id in a packed key: all 16 low bits under a bf16 logit, 8 under an fp32 one.
template <typename T>
constexpr int kIdBits = sizeof(T) == 2 ? 16 : 8;
template <typename T, int kThreads, int kN>
constexpr bool kPackable = kThreads == 32 && kThreads * kN <= (1 << kIdBits<T>);

// Sorts a thread's keys, largest first (Batcher's odd-even merge sort, all comparisons known at compile
// time).
template <int kN>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[kN]) {
#pragma unroll
    for (int p = 1; p < kN; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int j = k % p; j <= kN - 1 - k; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < kN && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = key[i + j], b = key[i + j + k];
                        key[i + j] = max(a, b);
                        key[i + j + k] = min(a, b);
                    }
}

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
    const T* z = logits + row * E;
    int32_t* my_ids = ids + row * K;
    float* my_scores = scores + row * K;
    uint32_t key[kN];
    load_keys<T, kThreads, kN, kVec>(z, E, t, key);
    float m = 0.0f, total = 0.0f;
    if (!normalize) {  // the sum of all exponentials, against the largest logit
        uint32_t best = 0u;
#pragma unroll
        for (int i = 0; i < kN; ++i) best = max(best, key[i]);
        m = key_value(red.argmax(best, t).x);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (key[i] != 0u) s += expf(key_value(key[i]) - m);
        total = red.sum(s);
    }
    int32_t id_k = 0;  // lane k % 32 keeps choice k until 32 of them are stored at once
    float part = 0.0f;
    // Choices first + lane of the first warp: their exponentials against the first choice, the largest.
    auto exponential = [&](int first) {
        const float v = first + t < K ? to_float(z[id_k]) : -INFINITY;
        if (first == 0) m = __shfl_sync(0xffffffffu, v, 0);
        const float e = expf(v - m);
        part += first + t < K ? e : 0.0f;
        return e;
    };
    auto store = [&](int first) {  // not yet scaled
        const float e = exponential(first);
        my_ids[first + t] = id_k;
        my_scores[first + t] = e;
    };
    bool exact = false;
    if constexpr (kPackable<T, kThreads, kN>) {
        constexpr uint32_t kIds = (1u << kIdBits<T>) - 1u;
#pragma unroll
        for (int i = 0; i < kN; ++i)  // equal logits: the lowest id is the largest key
            key[i] = key[i] == 0u ? 0u : (key[i] & ~kIds) | (kIds - expert_of<kThreads, kVec>(i, t));
        sort_keys<kN>(key);
        exact = true;
        uint32_t before = 0u;
        // fp32: one round more, to see that the last choice is clear of what comes after it
        const int rounds = sizeof(T) == 2 ? K : K + 1;
        for (int k = 0; k < rounds; ++k) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
            const bool mine = key[0] == best;
#pragma unroll
            for (int i = 0; i < kN - 1; ++i) key[i] = mine ? key[i + 1] : key[i];
            key[kN - 1] = mine ? 0u : key[kN - 1];
            if constexpr (sizeof(T) == 4) {
                exact = exact && (best ^ before) > kIds;
                before = best;
                if (k == K) break;
            }
            if (t == (k & 31)) id_k = static_cast<int32_t>(kIds - (best & kIds));
            if ((k & 31) == 31) store(k - 31);
        }
    }
    if (!exact) {  // the same for the whole warp or block
        load_keys<T, kThreads, kN, kVec>(z, E, t, key);
        part = 0.0f;
        for (int k = 0; k < K; ++k) {
            uint32_t best = 0u;
            int at = 0;
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (key[i] > best) best = key[i], at = i;
            const uint2 top = red.argmax(best, expert_of<kThreads, kVec>(at, t));
            if (t == (k & 31)) id_k = static_cast<int32_t>(top.y);
            const int own = static_cast<int>(top.y) - t * kVec;  // its place among this thread's, if it is one
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (own == expert_of<kThreads, kVec>(i, 0)) key[i] = 0u;
            if ((k & 31) == 31 && t < 32) store(k - 31);
        }
    }
    if (t >= 32) return;
    const int rest = K & ~31;  // choices [rest, K) are still in registers
    const bool mine = rest + t < K;
    const float e_k = rest < K ? exponential(rest) : 0.0f;
    if (normalize) total = warp_sum(part);
    const bool none = m == -INFINITY;  // a row with nothing but -inf has scores of 0
    const float inv = 1.0f / total;
    if (mine) {
        my_ids[rest + t] = id_k;
        my_scores[rest + t] = none ? 0.0f : e_k * inv;
    }
    for (int k = t; k < rest; k += 32) my_scores[k] = none ? 0.0f : my_scores[k] * inv;  // as this thread wrote it
}

// A lane owns each choice (k = t, t + kThreads, ...); an id outside [0, E) is none. The row is first written
// as if nothing were chosen, then the choices' own gradients over it.
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
    const T* zr = logits + row * E;
    T* dr = dlogits + row * E;
    const int32_t* my_ids = ids + row * K;
    const float* my_ds = dscores + row * K;
    auto inside = [&](int32_t id) { return id >= 0 && id < E; };
    float z[kN];
    uint32_t best = 0u;
    if (normalize) {
        for (int k = t; k < K; k += kThreads) {
            const int32_t id = __ldg(my_ids + k);
            if (inside(id)) best = max(best, order_key(to_float(zr[id])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; i += kVec) {
            const int e0 = expert_of<kThreads, kVec>(i, t);
            if (e0 < E) {
                const auto p = *reinterpret_cast<const LogitPack<T, kVec>*>(zr + e0);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    z[i + e] = to_float(p.v[e]);
                    best = max(best, order_key(z[i + e]));
                }
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) z[i + e] = -INFINITY;
            }
        }
    }
    const uint32_t top = red.argmax(best, t).x;
    const float m = top == 0u ? -INFINITY : key_value(top);
    const bool none = m == -INFINITY;  // nothing chosen, or everything masked: no gradient
    float s = 0.0f, dot = 0.0f;
    if (!normalize) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            z[i] = expf(z[i] - m);
            s += z[i];
        }
    }
    for (int k = t; k < K; k += kThreads) {
        const int32_t id = __ldg(my_ids + k);
        if (inside(id)) {
            const float e = expf(to_float(zr[id]) - m);
            if (normalize) s += e;
            dot += e * __ldg(my_ds + k);
        }
    }
    s = red.sum(s);
    dot = red.sum(dot);
    const float inv = 1.0f / s;
    dot *= inv;
#pragma unroll
    for (int i = 0; i < kN; i += kVec) {
        const int e0 = expert_of<kThreads, kVec>(i, t);
        if (e0 < E) {
            LogitPack<T, kVec> p;
#pragma unroll
            for (int e = 0; e < kVec; ++e) p.v[e] = from_float<T>(none || normalize ? 0.0f : z[i + e] * inv * -dot);
            *reinterpret_cast<LogitPack<T, kVec>*>(dr + e0) = p;
        }
    }
    // orders the row's stores before the choices' own, which other threads of the row make
    if constexpr (kThreads > 32) __syncthreads();
    else __syncwarp();
    for (int k = t; k < K; k += kThreads) {
        const int32_t id = __ldg(my_ids + k);
        if (inside(id))
            dr[id] = from_float<T>(none ? 0.0f : expf(to_float(zr[id]) - m) * inv * (__ldg(my_ds + k) - dot));
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
