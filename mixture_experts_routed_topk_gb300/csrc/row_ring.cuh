// row_ring.cuh -- what the norms over rows share: groups of threads that own a row, their sums, a ring of rows in
// shared memory that asynchronous copies fill, and the parameters in registers.
#pragma once

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "ptx_sm103.cuh"
#include "row_pieces.cuh"
#include "train_internal.cuh"

namespace moe {
namespace {

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

constexpr int kLnThreads = 512;
constexpr int kLnN = 16;  // elements of a row per thread

__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sums of kN (1, 2 or 4) values over the kGroup threads of a row; every thread of the group gets them.
// Lanes trade halves of the values as they add, so that after log2(kN) steps a lane carries one value:
// 5 or 6 shuffles for what would take 10 or 20. Each group has a named barrier; the two buffers
// alternate, so that one barrier per sum is enough: a warp writes buffer b again only after the barrier
// of the sum in between, which every reader has passed.
template <int kGroup, int kN>
struct GroupSum {
    static_assert(kN == 1 || kN == 2 || kN == 4, "values");
    static constexpr int kSpan = 32 / kN;  // lanes that end up with the same value
    float (*buf)[kN][kLnThreads / 32];
    int turn = 0;

    __device__ void operator()(float (&v)[kN]) {
        const int lane = threadIdx.x & 31;
        float t;
        {
            const bool up = lane & 16;
            if constexpr (kN == 4) {
                float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
                a += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
                b += __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
                const bool second = lane & 8;
                t = (second ? b : a) + __shfl_xor_sync(0xffffffffu, second ? a : b, 8);
            } else if constexpr (kN == 1) {
                t = v[0];
            } else {
                t = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
            }
        }
#pragma unroll
        for (int o = kSpan / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if constexpr (kGroup > 32) {
            constexpr int kWarps = kGroup / 32;
            const int group = threadIdx.x / kGroup, first = group * kWarps;
            float(&b)[kN][kLnThreads / 32] = buf[turn];
            turn ^= 1;
            if (lane % kSpan == 0) b[lane / kSpan][threadIdx.x >> 5] = t;
            group_barrier(1 + group, kGroup);
            // lane l adds value l / kSpan over the warps l % kSpan, l % kSpan + kSpan, ...
            t = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; w += kSpan)
                if (w + lane % kSpan < kWarps) t += b[lane / kSpan][first + w + lane % kSpan];
#pragma unroll
            for (int o = kSpan / 2; o > 0; o >>= 1)
                if (o < kWarps) t += __shfl_xor_sync(0xffffffffu, t, o);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = __shfl_sync(0xffffffffu, t, i * kSpan);
    }
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// One tensor's share of a ring stage: kLnThreads x kLnN elements, and 16 bytes more for each of up to 16
// rows, whose covering pieces may begin before and end after them.
template <typename T, int kN = kLnN>
constexpr int kTensorBytes = kLnThreads * kN * static_cast<int>(sizeof(T)) + 256;
// The covering pieces of one group's row.
template <typename T, int kGroup, int kN = kLnN>
constexpr int kPiecesBytes = kGroup * kN * static_cast<int>(sizeof(T)) + 16;

// A row as a group's threads see it in shared memory: element (i, e) of thread `lane` is element
// index(i, e) of the row.
template <typename T, int kGroup, bool kAligned, int kN = kLnN>
struct Row {
    static constexpr int kVec = kAligned ? 16 / static_cast<int>(sizeof(T)) : 1;
    static constexpr int kVecs = kN / kVec;

    __device__ static int index(int i, int lane) { return (i * kGroup + lane) * kVec; }

    // Starts the copies of row `row` of the tensor [rows, D] at base into this tensor's part of a stage.
    __device__ static void fetch(uint8_t* part, const T* base, int64_t row, int64_t rows, int32_t D, int lane) {
        if constexpr (kAligned) {
            const T* src = base + row * D;
            uint8_t* dst = part + 16 * static_cast<int>(threadIdx.x);
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (index(i, lane) < D) copy_async16(dst + i * kLnThreads * 16, src + index(i, lane));
        } else {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
            const uintptr_t hi = lo + static_cast<uintptr_t>(rows) * D * sizeof(T);
            const uintptr_t begin = lo + static_cast<uintptr_t>(row) * D * sizeof(T);
            const uintptr_t first = begin & ~static_cast<uintptr_t>(15);
            const int pieces = static_cast<int>((begin + D * sizeof(T) + 15 - first) / 16);
            uint8_t* dst = part + (threadIdx.x / kGroup) * kPiecesBytes<T, kGroup, kN>;
            for (int c = lane; c < pieces; c += kGroup) {
                const uintptr_t at = first + 16 * static_cast<uintptr_t>(c);
                if (at >= lo && at + 16 <= hi) {
                    copy_async16(dst + 16 * c, reinterpret_cast<const void*>(at));
                } else {  // the tensor's own first and last piece: only the elements inside it
                    for (uintptr_t a = at < lo ? lo : at; a < at + 16 && a < hi; a += sizeof(T))
                        *reinterpret_cast<T*>(dst + 16 * c + (a - at)) = *reinterpret_cast<const T*>(a);
                }
            }
        }
    }

    // Vector i of this thread's part of the row (index(i, lane) < D).
    __device__ static Pack<T, kVec> get(const uint8_t* part, const T* base, int64_t row, int32_t D, int i, int lane) {
        if constexpr (kAligned) {
            return *reinterpret_cast<const Pack<T, kVec>*>(part + 16 * (i * kLnThreads + static_cast<int>(threadIdx.x)));
        } else {
            const uintptr_t begin = reinterpret_cast<uintptr_t>(base) + static_cast<uintptr_t>(row) * D * sizeof(T);
            const uint8_t* r = part + (threadIdx.x / kGroup) * kPiecesBytes<T, kGroup, kN> + (begin & 15);
            return *reinterpret_cast<const Pack<T, kVec>*>(r + index(i, lane) * sizeof(T));
        }
    }
};

// This thread's parameters, in the order of its elements.
template <class R, int kN>
__device__ __forceinline__ void load_params(const Param& a, int32_t D, int lane, float none, float (&out)[kN]) {
    static_assert(R::kVec * R::kVecs == kN, "elements");
#pragma unroll
    for (int i = 0; i < R::kVecs; ++i) {
        float t[R::kVec];
#pragma unroll
        for (int e = 0; e < R::kVec; ++e) t[e] = none;
        if (R::index(i, lane) < D) load_param<R::kVec>(a, R::index(i, lane), none, t);
#pragma unroll
        for (int e = 0; e < R::kVec; ++e) out[i * R::kVec + e] = t[e];
    }
}

// Elements of a row per thread in the norms around a block, and the longest row that a group holds.
template <typename T>
constexpr int kBnN = sizeof(T) == 4 ? 8 : 16;
template <typename T>
constexpr int kBnMaxHeldD = kLnThreads * kBnN<T>;

template <typename T>
__device__ __forceinline__ void store_two(T* to, float2 v) {
    to[0] = from_float<T>(v.x);
    to[1] = from_float<T>(v.y);
}
template <>
__device__ __forceinline__ void store_two<__nv_bfloat16>(__nv_bfloat16* to, float2 v) {
    *reinterpret_cast<__nv_bfloat162*>(to) = __float22bfloat162_rn(v);
}
template <>
__device__ __forceinline__ void store_two<__half>(__half* to, float2 v) {
    *reinterpret_cast<__half2*>(to) = __float22half2_rn(v);
}

// A thread's share of a row in chunks of 16 bytes, as pairs of floats for the instructions that take two. A lane
// copies and reads only its own chunks.
//
// kWhole: every row starts and ends on 16-byte boundaries. Otherwise the chunks are the 16-byte pieces of memory that
// cover the row, so that rows of any length come and go in 16-byte accesses: the first and last may hold neighbours'
// elements, which count as 0 and are not written. All tensors have to lie the same way to those pieces, and a
// group's rows too: `lead` is how many elements of the first piece come before the row.
template <typename T, int kGroup, bool kWhole, int kN>
struct Cells {
    static constexpr int kC = 16 / static_cast<int>(sizeof(T)), kPairs = kC / 2, kChunks = kN / kC;
    // Whether rows may be shorter than a piece. A larger group has rows of nearly half its elements or more.
    static constexpr bool kShort = kGroup == 32;
    static_assert(kGroup == 32 || kGroup * kN / 2 >= 2 * kC, "rows of a piece or more");
    using Pairs = float2[kPairs];
    int lane, lead;
    int32_t D;

    // base: any of the tensors; row: any of the group's rows.
    __device__ Cells(const T* base, int64_t row, int32_t d, int l) : lane(l), lead(0), D(d) {
        if constexpr (!kWhole) {
            lead = static_cast<int>((reinterpret_cast<uintptr_t>(base) / sizeof(T) + static_cast<uintptr_t>(row) * d) % kC);
            // Hidden from the compiler's optimizer, which otherwise relates it to the lane: with nvcc 13.0 stores to
            // own[index(c, e)] in shared memory under has(c, e), own being the group's part of it, then went to the first
            // group's part for the chunks that are not whole. A kernel of nothing but such stores, with chunks of eight
            // elements, does it too, as inline assembly as well; not with chunks of four, with global memory, or with
            // -Xcicc -O1 (-Xptxas -O0 changes nothing).
            asm volatile("" : "+r"(lead));
        }
    }
    // The element of the row that is element e of chunk c.
    __device__ int index(int c, int e) const { return (c * kGroup + lane) * kC + e - (kWhole ? 0 : lead); }
    __device__ bool any(int c) const { return index(c, 0) < D; }
    __device__ bool has(int c, int e) const { return index(c, e) >= 0 && index(c, e) < D; }
    __device__ bool whole(int c) const { return kWhole || (index(c, 0) >= 0 && index(c, kC - 1) < D); }

    __device__ void fetch(uint8_t* part, const T* base, int64_t row, int64_t rows) const {
        uint8_t* dst = part + 16 * static_cast<int>(threadIdx.x);
        const T* src = base + row * D;
        if (kWhole || (row > 0 && row < rows - 1 && neighbours_cover<kShort>(D, kC))) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                if (any(c)) copy_async16(dst + c * kLnThreads * 16, src + index(c, 0));
        } else {  // before the tensor's first element and after its last there is nothing to read
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                if (!any(c)) continue;
                if (piece_inside<kShort>(row, rows, D, index(c, 0), index(c, kC - 1))) {
                    copy_async16(dst + c * kLnThreads * 16, src + index(c, 0));
                } else {
                    for (int e = 0; e < kC; ++e)
                        if (has(c, e)) reinterpret_cast<T*>(dst + c * kLnThreads * 16)[e] = src[index(c, e)];
                }
            }
        }
    }
    // Once the row is there: zeros for the neighbours' elements in the lane's chunks.
    __device__ void trim(uint8_t* part) const {
        if constexpr (!kWhole) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (!any(c) || whole(c)) continue;
                auto* at = reinterpret_cast<Pack<T, kC>*>(part + 16 * (c * kLnThreads + static_cast<int>(threadIdx.x)));
                auto p = *at;
#pragma unroll
                for (int e = 0; e < kC; ++e)
                    if (!has(c, e)) p.v[e] = from_float<T>(0.0f);
                *at = p;
            }
        }
    }
    // The lane's chunk c (any(c)) of a row that has been trimmed.
    __device__ void get(const uint8_t* part, int c, Pairs& v) const {
        const auto p = *reinterpret_cast<const Pack<T, kC>*>(part + 16 * (c * kLnThreads + static_cast<int>(threadIdx.x)));
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[i] = make_float2(to_float(p.v[2 * i]), to_float(p.v[2 * i + 1]));
    }
    __device__ void put(T* base, int64_t row, int c, const Pairs& v) const {
        T* to = base + row * D;
        if (kWhole || whole(c)) {
            Pack<T, kC> p;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) store_two(p.v + 2 * i, v[i]);
            *reinterpret_cast<Pack<T, kC>*>(to + index(c, 0)) = p;
        } else {
#pragma unroll
            for (int e = 0; e < kC; ++e)
                if (has(c, e)) to[index(c, e)] = from_float<T>(e % 2 ? v[e / 2].y : v[e / 2].x);
        }
    }
    // The lane's parameters, in the order of its elements.
    __device__ void params(const Param& a, float none, float2 (&out)[kN / 2]) const {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float t[kC];
            if (kWhole) {
#pragma unroll
                for (int e = 0; e < kC; ++e) t[e] = none;
                if (any(c)) load_param<kC>(a, index(c, 0), none, t);
            } else {
#pragma unroll
                for (int e = 0; e < kC; ++e) {
                    float one[1] = {none};
                    if (has(c, e)) load_param<1>(a, index(c, e), none, one);
                    t[e] = one[0];
                }
            }
#pragma unroll
            for (int i = 0; i < kPairs; ++i) out[c * kPairs + i] = make_float2(t[2 * i], t[2 * i + 1]);
        }
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Bytes of a tensor's row in a stage of the ring: what a group of all threads needs, or all groups' together.
template <typename T, int kGroup>
int tensor_stride(int32_t D) {
    constexpr int kC = 16 / static_cast<int>(sizeof(T));
    const int full = kTensorBytes<T, kBnN<T>>;
    return kGroup < kLnThreads ? full : std::min(full, (static_cast<int>(ceil_div(D, kC)) + 2) * 16);
}

// Blocks of a grid whose groups keep their rows' way of lying to 16-byte pieces: the stride between a group's rows is
// a multiple of eight, or each has but one.
inline int64_t row_blocks(int64_t rows, int rows_per_block, int64_t most) {
    const int64_t need = ceil_div(rows, rows_per_block);
    return need <= most ? need : most / 8 * 8;
}

// Whether the tensors lie the same way to 16-byte pieces of memory (null ones lie any way).
inline bool lie_alike(std::initializer_list<const void*> tensors) {
    const void* first = nullptr;
    for (const void* t : tensors) {
        if (t && !first) first = t;
        if (t && (reinterpret_cast<uintptr_t>(t) ^ reinterpret_cast<uintptr_t>(first)) % 16 != 0) return false;
    }
    return true;
}

bool rows_aligned16(const void* p, int64_t row_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0;
}

Param param(const void* p, int32_t dtype) { return Param{p, dtype, reinterpret_cast<uintptr_t>(p) % 16 == 0}; }

// Allows the kernel its dynamic shared memory, once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

}  // namespace
}  // namespace moe
