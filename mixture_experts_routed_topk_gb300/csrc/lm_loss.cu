// lm_loss.cu -- losses of a linear head over a large vocabulary, without keeping its logits:
// softmax cross entropy, and distillation from a teacher's top logits. Forward and backward.
//
// For hidden rows x [T, D] and head weights W [V, D], with u = 1 / temperature (1 for cross entropy):
//   z = u x W^T                                     [T, V], never stored
//   lse_t = log sum_v exp(z_tv),   q = exp(z - lse)
//   a row's targets are K pairs (vocabulary id, probability p): the label with p = 1, or the softmax
//   of the teacher's kept logits at the temperature
//   cross entropy  loss_t = lse_t - z_t,target
//   distillation   loss_t = tau^2 sum_j p_j (log p_j - (z_tj - lse_t))
//   backward       dl = c_t (q - sum_j p_j onehot_j),  c_t = dloss_t (cross entropy), tau dloss_t
//                  dx = dl W,  dW = dl^T x
// A row whose label is ignored, or none of whose teacher entries is kept, has loss 0 and c_t = 0.
//
// All products run on the tcgen05 pipeline of gemm_pipeline.cuh (bf16 operands, fp32 accumulation):
//   forward: the epilogue reduces a logit tile of 128 rows and 32 to 256 columns (pick_columns) to one
//     (maximum, sum of exponentials) per row and picks the targets' logits out of it; k_lm_join joins a
//     row's tiles.
//   backward: over pieces of the vocabulary that fit the workspace, the epilogue of the recomputed
//     logits writes dl in bf16; one more grid turns the piece into its rows of dW and its share of
//     dx. dx is summed over pieces and over slices of the contraction in fp32 and rounded once.
// Rounding dl to bf16 costs each term of dx and dW at most half a bf16 step, as much as rounding
// the results; it is what lets the two products use the bf16 tensor cores.
//
// A row's targets are first sorted by id (k_lm_teacher), so that a tile finds its own with one
// search, and each thread picks them out of the 32 logits that it holds in registers. Ids that repeat
// in a row count once each, in order.
//
// Measured, calls back to back (cuBLAS's bf16 rate is 1915 TFLOP/s in bursts, 1717 sustained): 4096 x 2048 x
// 32000 (T x D x V) forward 307 us (1749 TFLOP/s), backward 1003 us (1605), 1045 us (1541) as a loop of calls
// on changing inputs sees it. The backward's shares are 32 % dl, 35 % dx and 33 % dW, with the tensor pipe 78, 84
// and 84 % busy; 85 % in the forward, whose exponentials run under the next tile's products.
// 16 x 2048 x 32000 forward 32 us: some 26 us of it read W's 131 MB. 64 x 2048 x 32000 backward 85 us, where
// the traffic takes 39: dl's 125 tiles leave 27 SMs idle, and W is read from memory twice, once for the logits
// and again for dx, as it does not fit L2 beside what is written.
#include <algorithm>
#include <climits>

#include "gemm_pipeline.cuh"
#include "train_internal.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kNoTarget = INT_MAX;
constexpr int kLmMaxK = 256;

// 2^x through the hardware (at most 2 units in the last place; results below 2^-126 are 0).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The same with subnormal results: a probability below 2^-126 still has a gradient where it meets
// large hidden values.
__device__ __forceinline__ float exp2_full(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------------------------------ targets

// Distillation: one warp per row. sid / sp: the kept ids in ascending order (equal ids in the order
// given) with their probabilities, then kNoTarget / 0. ent[t] = sum_j p_j log p_j. coef[t] = tau dloss[t], or 0
// for a row without a distribution (backward only).
// An entry with a negative id is not kept (its logit is not looked at). The row's largest logit is taken off
// before the temperature divides: logits near the ends of their type would overflow under one below 1.
__global__ void __launch_bounds__(128)
    k_lm_teacher(const int32_t* __restrict__ ids, const float* __restrict__ logits, int64_t T, int32_t K, int32_t V,
                 float inv_tau, float tau, const float* __restrict__ dloss, int32_t* __restrict__ sid,
                 float* __restrict__ sp, float* __restrict__ ent, float* __restrict__ coef,
                 uint32_t* __restrict__ status) {
    __shared__ int32_t s_id[4][kLmMaxK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + warp;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= T) return;  // whole warps
    int32_t* row_id = s_id[warp];
    float a[kLmMaxK / 32];
    float m = -INFINITY;
    int kept = 0;
    bool bad = false, nan = false;
#pragma unroll
    for (int i = 0; i < kLmMaxK / 32; ++i) {
        const int j = i * 32 + lane;
        a[i] = -INFINITY;
        if (j < K) {
            const int32_t id = __ldg(ids + t * K + j);
            const bool ok = id >= 0 && id < V;
            bad = bad || id >= V;
            row_id[j] = ok ? id : kNoTarget;
            if (ok) {
                a[i] = __ldg(logits + t * K + j);
                nan = nan || a[i] != a[i];
                m = fmaxf(m, a[i]);
                ++kept;
            }
        }
    }
    if (bad) atomicOr(status, MOE_DEV_BAD_TARGET);
    __syncwarp();
    nan = __any_sync(0xffffffffu, nan);
    kept = __reduce_add_sync(0xffffffffu, kept);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // kept entries of -inf only have no distribution: the row counts as one without entries
    const bool none = kept == 0 || (m == -INFINITY && !nan);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kLmMaxK / 32; ++i) {
        a[i] = (a[i] - m) * inv_tau;
        s += none ? 0.0f : expf(a[i]);
    }
    s = warp_sum(s);
    const float log_s = logf(s);
    float e = 0.0f;
#pragma unroll
    for (int i = 0; i < kLmMaxK / 32; ++i) {
        const int j = i * 32 + lane;
        if (j < K) {
            const int32_t id = none ? kNoTarget : row_id[j];
            const bool ok = id != kNoTarget;
            const float p = ok ? expf(a[i]) / s : 0.0f;
            if (ok && p != 0.0f) e += p * (a[i] - log_s);
            int rank = 0;
            for (int l = 0; l < K; ++l) {
                const int32_t other = none ? kNoTarget : row_id[l];
                rank += (other < id || (other == id && l < j)) ? 1 : 0;
            }
            sid[t * K + rank] = id;
            sp[t * K + rank] = p;
        }
    }
    e = warp_sum(e);
    if (lane == 0) {
        ent[t] = e;
        if (coef) coef[t] = none ? 0.0f : tau * dloss[t];
    }
}

// ------------------------------------------------------------------------------- tile policies

struct LmArgs : GemmArgs {
    int64_t T;
    int32_t V;           // vocabulary (columns at and past it do not exist)
    int32_t v0;          // first column of the piece
    int32_t group;       // row tiles walked together along the columns
    int32_t bn;          // columns per logit tile (a multiple of 32, at most 256)
    int32_t bm;          // rows of x (or dl) that a tile loads (box_rows)
    int32_t K;           // targets per row
    const int32_t* sid;  // [T, K] sorted target ids
    const float* sp;     // [T, K] their probabilities; null: 1
    float* zt;           // [T, K] out: the targets' accumulators
    float2* part;        // [ntiles][T] out: the tile's largest accumulator, and the sum of its exponentials against it
    float scale2;        // accumulator to scaled logit (logit_scale) in units of log 2, for base-2 exponentials
    const float* lse;    // [T]
    const float* coef;   // [T] distillation: the factor of the row's dl
    const float* dloss;  // [T] cross entropy: the same, where the label counts
    int32_t ignore_index;
    int32_t pitch;       // row length of the dl piece
    int32_t kb_slice;    // K steps per slice of the contraction (dx)
    bool accumulate;     // dx: add to the slice's sums instead of starting them
    bool direct;         // dx: one slice and one piece, so the tile is the result
    // the gradients' grid: dx tiles (all slices), then dW's tiles with their own counts
    int32_t dx_tiles, dw_tiles;
    int32_t dw_mtiles, dw_kblocks, dw_group;
};

struct LmTile {
    int32_t m, n, kblocks, slice, bn, bm;
    bool dw;
};

// Row tiles in groups; within a group columns outermost, so that a group's rows of A stay
// in L2 while B streams by once per group.
__device__ __forceinline__ void grouped_mn(int32_t tile, int32_t group, int32_t mtiles, int32_t ntiles, LmTile* t) {
    const int32_t per_group = group * ntiles;
    const int32_t g = tile / per_group;
    const int32_t r = tile - g * per_group;
    const int32_t rows = min(group, mtiles - g * group);
    t->n = r / rows;
    t->m = g * group + r - t->n * rows;
}

// The row's first sorted target at or past vocabulary id `first`.
__device__ __forceinline__ int first_target(const int32_t* sid, int32_t K, int32_t first) {
    int lo = 0, hi = K;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(sid + mid) < first) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Stores 128 bytes of each of the warp's 32 rows, `pitch` bytes apart from base on (the first `live` of
// them): through the staging rows, so that each store instruction writes four whole 128-byte segments.
__device__ __forceinline__ void store_rows(uint4* stage, const uint32_t (&words)[32], char* base, int64_t pitch,
                                           int live) {
    const int lane = threadIdx.x & 31;
    uint4* mine = stage + lane * kStageRowU4;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        mine[c] = make_uint4(words[4 * c], words[4 * c + 1], words[4 * c + 2], words[4 * c + 3]);
    __syncwarp();
    char* dst = base + (lane >> 3) * pitch + 16 * (lane & 7);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (4 * j + (lane >> 3) < live)
            *reinterpret_cast<uint4*>(dst + 4 * j * pitch) = stage[(4 * j + (lane >> 3)) * kStageRowU4 + (lane & 7)];
    __syncwarp();
}

// The warp's 32 rows of a 128 x 256 accumulator as bf16: columns [0, cols) (cols a multiple of 64) to rows
// `pitch` elements apart from base on. The next 64 columns leave tensor memory while these are stored.
__device__ __forceinline__ void store_tile_bf16(uint32_t taddr, uint4* stage, __nv_bfloat16* base, int64_t pitch,
                                                int32_t cols, int live) {
    uint32_t v0[32], v1[32];
    __syncwarp();
    tmem_ld_32cols(taddr, v0);
    tmem_ld_32cols(taddr + 32, v1);
#pragma unroll 1
    for (int32_t c = 0; c < cols; c += 64) {
        tmem_ld_wait(v0);
        tmem_ld_tie(v1);
        uint32_t words[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            words[i] = pack_bf16x2(__uint_as_float(v0[2 * i]), __uint_as_float(v0[2 * i + 1]));
            words[16 + i] = pack_bf16x2(__uint_as_float(v1[2 * i]), __uint_as_float(v1[2 * i + 1]));
        }
        if (c + 64 < cols) {
            tmem_ld_32cols(taddr + c + 64, v0);
            tmem_ld_32cols(taddr + c + 96, v1);
        }
        store_rows(stage, words, reinterpret_cast<char*>(base + c), 2 * pitch, live);
    }
}

// Rows of the warp's 32, from `first` on, that lie below `limit`.
__device__ __forceinline__ int live_rows(int64_t first, int64_t limit) {
    const int64_t n = limit - first;
    return n >= 32 ? 32 : n > 0 ? static_cast<int>(n) : 0;
}

// A = x rows, B = W rows, both K-major; K = D.
struct LmLogits {
    using Args = LmArgs;
    using Tile = LmTile;
    static constexpr bool kAMnMajor = false, kBMnMajor = false;
    static constexpr uint32_t kIdesc = idesc_bf16_f32(kBM, kBRows);

    __device__ static int32_t num_tiles(const Args& a) { return a.mtiles * a.ntiles; }
    __device__ static Tile decode(int32_t tile, const Args& a) {
        Tile t{};
        grouped_mn(tile, a.group, a.mtiles, a.ntiles, &t);
        t.kblocks = a.kblocks;
        t.bn = a.bn;
        t.bm = a.bm;
        return t;
    }
    __device__ static uint32_t idesc(const Tile& t) {
        return (kIdesc & ~(63u << 17)) | (static_cast<uint32_t>(t.bn >> 3) << 17);
    }
    __device__ static uint32_t tx_bytes(const Tile& t) { return (t.bm + t.bn) * kBK * 2; }
    __device__ static void load(const Tile& t, int32_t kb, uint8_t* sa, uint8_t* sb, uint64_t* bar,
                                const CUtensorMap* ta, const CUtensorMap* tb, const Args& a) {
        tma_load_2d(sa, ta, bar, kb * kBK, t.m * kBM);
        tma_load_2d(sb, tb, bar, kb * kBK, a.v0 + t.n * a.bn);
    }
};

// Forward: a tile's share of the row's softmax sum, and the targets' logits. Both the maximum and the targets
// are kept as the accumulators they are, and exponentials are taken of differences to the maximum: the largest
// term is then exactly 1 and the sum 1 or more, and a target that is the maximum is exactly 0 below it, however
// large the logit. With each scaled and rounded for itself, a row that is sure of its target would get a loss
// off by roundings of the logit's size, and below 0 as often as not.
struct LmLse : LmLogits {
    __device__ static void epilogue(const Tile& t, uint32_t taddr, int row_in_tile, uint4*, const Args& a) {
        const int64_t row = static_cast<int64_t>(t.m) * kBM + row_in_tile;
        const bool live = row < a.T;
        const int32_t n0 = t.n * t.bn;
        const float scale2 = a.scale2;
        int j = 0;
        int32_t next = kNoTarget;
        const int32_t* sid = a.sid + row * a.K;
        if (live) {
            j = first_target(sid, a.K, n0);
            if (j < a.K) next = __ldg(sid + j);
        }
        float m = -INFINITY, s = 0.0f;
#pragma unroll 1
        for (int c = 0; c < t.bn / 32; ++c) {
            const int32_t c0 = n0 + 32 * c;
            if (c0 >= a.V) break;  // warp-uniform
            __syncwarp();
            uint32_t w[32];
            tmem_ld_32cols(taddr + 32 * c, w);
            tmem_ld_wait(w);
            if (c0 + 32 > a.V) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c0 + i >= a.V) w[i] = __float_as_uint(-INFINITY);
            }
            while (next < c0 + 32) {
                uint32_t z = 0u;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (next == c0 + i) z = w[i];
                a.zt[row * a.K + j] = __uint_as_float(z);
                ++j;
                next = j < a.K ? __ldg(sid + j) : kNoTarget;
            }
            float cm = __uint_as_float(w[0]);
#pragma unroll
            for (int i = 1; i < 32; ++i) cm = fmaxf(cm, __uint_as_float(w[i]));
            const float top = fmaxf(m, cm);
            const float base = top == -INFINITY ? 0.0f : top;  // nothing but -inf so far: its terms are 0
            // small terms meet each other before they meet the 1; two numbers to an instruction
            float2 q[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 z = make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
                const float2 d = __fmul2_rn(__fadd2_rn(z, make_float2(-base, -base)), make_float2(scale2, scale2));
                q[(i >> 1) & 1] = __fadd2_rn(q[(i >> 1) & 1], make_float2(exp2_fast(d.x), exp2_fast(d.y)));
            }
            s = fmaf(s, exp2_fast((m - base) * scale2), (q[0].x + q[0].y) + (q[1].x + q[1].y));
            m = top;
        }
        if (live) a.part[static_cast<int64_t>(t.n) * a.T + row] = make_float2(m, s);
    }
};

// Backward: the tile's dl in bf16 into the piece [T, pitch]; columns past the vocabulary get zeros.
struct LmDlogits : LmLogits {
    __device__ static void epilogue(const Tile& t, uint32_t taddr, int row_in_tile, uint4* stage, const Args& a) {
        const int lane = threadIdx.x & 31;
        const int64_t row = static_cast<int64_t>(t.m) * kBM + row_in_tile;
        const bool live = row < a.T;
        const int32_t n0 = a.v0 + t.n * kBN2;
        const float scale2 = a.scale2;
        float coef = 0.0f, lse2 = 0.0f;
        int j = 0;
        int32_t next = kNoTarget;
        const int32_t* sid = a.sid + row * a.K;
        if (live) {
            lse2 = __ldg(a.lse + row) * kLog2e;
            if (a.sp == nullptr) {  // the labels as the caller gave them
                const int32_t id = __ldg(sid);
                const bool inside = id >= 0 && id < a.V, ignored = id == a.ignore_index;
                if (!inside && !ignored && n0 == 0) atomicOr(a.status, MOE_DEV_BAD_TARGET);
                if (inside && !ignored) {
                    coef = __ldg(a.dloss + row);
                    if (id >= n0) next = id;
                }
            } else {
                coef = __ldg(a.coef + row);
                j = first_target(sid, a.K, n0);
                if (j < a.K) next = __ldg(sid + j);
            }
        }
        const bool zero = coef == 0.0f;
#pragma unroll 1
        for (int cp = 0; cp < kBN2 / 64; ++cp) {
            uint32_t words[32];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int32_t c0 = n0 + 64 * cp + 32 * half;
                __syncwarp();
                uint32_t w[32];
                tmem_ld_32cols(taddr + 64 * cp + 32 * half, w);
                tmem_ld_wait(w);
                float d[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    d[i] = coef * exp2_full(fmaf(__uint_as_float(w[i]), scale2, -lse2));
                    if (zero || c0 + i >= a.V) d[i] = 0.0f;
                }
                while (next < c0 + 32) {
                    const float p = coef * (a.sp ? __ldg(a.sp + row * a.K + j) : 1.0f);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (next == c0 + i) d[i] -= p;
                    ++j;
                    next = j < a.K ? __ldg(sid + j) : kNoTarget;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) words[16 * half + i] = pack_bf16x2(d[2 * i], d[2 * i + 1]);
            }
            __syncwarp();
            store_rows(stage, words, reinterpret_cast<char*>(a.out0 + (row - lane) * a.pitch + t.n * kBN2 + 64 * cp),
                       2ll * a.pitch, live_rows(row - lane, a.T));
        }
    }
};

// The gradients of a piece:
//   dx:  A = dl piece rows (K-major, K = the piece's columns or a slice of them), B = W read MN-major as
//        B[n = d][k = v]
//   dW:  A = dl^T (MN-major: vocabulary contiguous), B = x (MN-major: d contiguous); K = T. TMA returns
//        zeros for rows past T, so the contraction needs no padding.
// kTogether: both in one grid, dx's tiles, the long ones, first; SMs take tiles as they get free, so that
// those that finish early go on with the other gradient. Otherwise one of the two, SMs in step.
template <bool kTogether>
struct LmGrads {
    using Args = LmArgs;
    using Tile = LmTile;
    static constexpr bool kBMnMajor = true;
    static constexpr uint32_t kIdesc = idesc_bf16_f32(kBM, kBRows, false, true);
    static constexpr bool kDynamicSchedule = kTogether;

    __device__ static int32_t num_tiles(const Args& a) { return a.dx_tiles + a.dw_tiles; }
    __device__ static Tile decode(int32_t tile, const Args& a) {
        Tile t{};
        t.bn = kBN2;
        t.dw = tile >= a.dx_tiles;
        if (t.dw) {
            grouped_mn(tile - a.dx_tiles, a.dw_group, a.dw_mtiles, a.ntiles, &t);
            t.kblocks = a.dw_kblocks;
            t.bm = kBM;
        } else {
            const int32_t per_slice = a.mtiles * a.ntiles;
            t.slice = tile / per_slice;
            grouped_mn(tile - t.slice * per_slice, a.group, a.mtiles, a.ntiles, &t);
            t.kblocks = min(a.kb_slice, a.kblocks - t.slice * a.kb_slice);
            t.bm = a.bm;
        }
        return t;
    }
    __device__ static bool a_mn_major(const Tile& t) { return t.dw; }
    __device__ static uint32_t idesc(const Tile& t) {
        return t.dw ? idesc_bf16_f32(kBM, kBRows, true, true) : kIdesc;
    }
    __device__ static uint32_t tx_bytes(const Tile& t) { return (t.bm + kBN2) * kBK * 2; }
    // maps: 0 dl rows, 1 W (64-wide boxes), 2 dl (64-wide boxes), 3 x (64-wide boxes)
    __device__ static void load(const Tile& t, int32_t kb, uint8_t* sa, uint8_t* sb, uint64_t* bar,
                                const CUtensorMap* ta, const CUtensorMap* tb, const Args& a) {
        if (t.dw) {
#pragma unroll
            for (int j = 0; j < kBM / 64; ++j)
                tma_load_2d(sa + j * kMnBoxBytes, ta + 2, bar, t.m * kBM + 64 * j, kb * kBK);
#pragma unroll
            for (int j = 0; j < kBRows / 64; ++j)
                tma_load_2d(sb + j * kMnBoxBytes, ta + 3, bar, t.n * kBN2 + 64 * j, kb * kBK);
            return;
        }
        const int32_t k = (t.slice * a.kb_slice + kb) * kBK;
        tma_load_2d(sa, ta, bar, k, t.m * kBM);
#pragma unroll
        for (int j = 0; j < kBRows / 64; ++j)
            tma_load_2d(sb + j * kMnBoxBytes, tb, bar, t.n * kBN2 + 64 * j, a.v0 + k);
    }
    __device__ static void epilogue(const Tile& t, uint32_t taddr, int row_in_tile, uint4* stage, const Args& a) {
        if (t.dw) {
            const int64_t v = static_cast<int64_t>(a.v0) + t.m * kBM + row_in_tile - (threadIdx.x & 31);
            const int32_t d0 = t.n * kBN2;
            store_tile_bf16(taddr, stage, a.out1 + v * a.D + d0, a.D, min(kBN2, a.D - d0), live_rows(v, a.V));
            return;
        }
        const int lane = threadIdx.x & 31;
        const int64_t row0 = static_cast<int64_t>(t.m) * kBM + row_in_tile - lane;  // the warp's first
        const int live = live_rows(row0, a.T);
        const int32_t d_tile = t.n * kBN2;
        if (a.direct) {
            store_tile_bf16(taddr, stage, a.out0 + row0 * a.D + d_tile, a.D, min(kBN2, a.D - d_tile), live);
            return;
        }
        float* sums = a.fout + static_cast<int64_t>(t.slice) * a.T * a.D;
#pragma unroll 1
        for (int c = 0; c < kBN2 / 32; ++c) {
            const int32_t d0 = d_tile + 32 * c;
            if (d0 >= a.D) break;  // warp-uniform
            uint32_t before[32];
            if (a.accumulate) {  // this warp's 32 rows of 32 sums, in whole 128-byte row segments
                uint4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int64_t r = row0 + 4 * q + (lane >> 3);
                    v[q] = r < a.T ? __ldcg(reinterpret_cast<const uint4*>(sums + r * a.D + d0) + (lane & 7))
                                   : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) stage[(4 * q + (lane >> 3)) * kStageRowU4 + (lane & 7)] = v[q];
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint4 x = stage[lane * kStageRowU4 + q];
                    before[4 * q] = x.x, before[4 * q + 1] = x.y, before[4 * q + 2] = x.z, before[4 * q + 3] = x.w;
                }
            }
            __syncwarp();
            uint32_t w[32];
            tmem_ld_32cols(taddr + 32 * c, w);
            tmem_ld_wait(w);
            if (a.accumulate) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    w[i] = __float_as_uint(__uint_as_float(w[i]) + __uint_as_float(before[i]));
            }
            store_rows(stage, w, reinterpret_cast<char*>(sums + row0 * a.D + d0), 4ll * a.D, live);
        }
    }
};

// --------------------------------------------------------------------------------- reductions

// Joins a row's tiles and forms its loss. A block owns 32 rows, one per lane; its warps take the
// tiles in turn and meet in shared memory in warp order. Then (distillation) each warp sums the targets
// of two rows. sp null: cross entropy, where sid holds the labels as the caller gave them.
// With the row's largest accumulator m and s = sum exp(z - m): a target's -log q is (m - its accumulator),
// scaled, plus log s. Both are 0 or more.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps)
    k_lm_join(const float2* __restrict__ part, int32_t ntiles, int64_t T, int32_t K, const int32_t* __restrict__ sid,
              const float* __restrict__ sp, const float* __restrict__ zt, const float* __restrict__ ent, float tau,
              float zscale, float scale2, int32_t ignore_index, int32_t V, float* __restrict__ loss,
              float* __restrict__ lse_out, uint32_t* __restrict__ status) {
    __shared__ float2 acc[kJoinWarps][32];
    __shared__ float2 s_row[32];  // the row's largest accumulator and log s
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    griddep_wait();
    griddep_launch_dependents();
    float m = -INFINITY, s = 0.0f;
    if (row < T) {
        auto add = [&](const float2& p) {
            const float top = fmaxf(m, p.x);
            s = (s == 0.0f ? 0.0f : s * exp2_fast((m - top) * scale2)) +
                (p.y == 0.0f ? 0.0f : p.y * exp2_fast((p.x - top) * scale2));
            m = top;
        };
        int n = warp;
        for (; n + 3 * kJoinWarps < ntiles; n += 4 * kJoinWarps) {
            float2 p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) p[u] = part[static_cast<int64_t>(n + u * kJoinWarps) * T + row];
#pragma unroll
            for (int u = 0; u < 4; ++u) add(p[u]);
        }
        for (; n < ntiles; n += kJoinWarps) add(part[static_cast<int64_t>(n) * T + row]);
    }
    acc[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp == 0 && row < T) {
        float top = acc[0][lane].x;
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, acc[w][lane].x);
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w)
            if (acc[w][lane].y != 0.0f) s += acc[w][lane].y * exp2_fast((acc[w][lane].x - top) * scale2);
        const float log_s = logf(s);
        lse_out[row] = fmaf(top, zscale, log_s);
        s_row[lane] = make_float2(top, log_s);
        if (sp == nullptr) {
            const int32_t id = sid[row];
            const bool inside = id >= 0 && id < V, ignored = id == ignore_index;
            if (!inside && !ignored) atomicOr(status, MOE_DEV_BAD_TARGET);
            loss[row] = inside && !ignored ? fmaf(top - zt[row], zscale, log_s) : 0.0f;
        }
    }
    if (sp == nullptr) return;
    __syncthreads();
    for (int r = warp; r < 32; r += kJoinWarps) {
        const int64_t t = static_cast<int64_t>(blockIdx.x) * 32 + r;
        if (t >= T) break;
        const float2 top_log = s_row[r];
        float l = 0.0f;
        bool any = false;
        for (int j = lane; j < K; j += 32) {
            if (sid[t * K + j] == kNoTarget) break;  // sorted: nothing after it
            any = true;
            const float p = sp[t * K + j];
            if (p != 0.0f) l += p * fmaf(top_log.x - zt[t * K + j], zscale, top_log.y);
        }
        __syncwarp();
        l = warp_sum(l);
        any = __any_sync(0xffffffffu, any);
        if (lane == 0) loss[t] = any ? tau * tau * (ent[t] + l) : 0.0f;
    }
}

// dx = bf16( sum over slices in slice order ).
__global__ void __launch_bounds__(256) k_lm_sum_slices(const float4* __restrict__ sums, int32_t slices, int64_t n4,
                                                       uint2* __restrict__ dx) {
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n4;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        float4 a = sums[i];
        int s = 1;
        for (; s + 7 < slices; s += 8) {  // eight loads at a time, added in slice order
            float4 b[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) b[u] = sums[(s + u) * n4 + i];
#pragma unroll
            for (int u = 0; u < 8; ++u) a.x += b[u].x, a.y += b[u].y, a.z += b[u].z, a.w += b[u].w;
        }
        for (; s < slices; ++s) {
            const float4 b = sums[s * n4 + i];
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        }
        dx[i] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    }
}

// ---------------------------------------------------------------------------------------- plan

constexpr size_t kRegionAlign = 256;
constexpr int kPlanSms = 152;                 // SMs of the GB300, for sizes that must not depend on the device
constexpr int64_t kPieceBytes = 512ll << 20;  // most bytes of one dl piece
constexpr int32_t kMinPiece = 2048;           // but at least this many columns
constexpr int kFirstTicket = 32;              // word of the workspace with the first piece's tile counter

struct LmPlan {
    int32_t mtiles, ntiles;  // of the logits, in 128 x 256 tiles
    int32_t fwd_bn, fwd_ntiles;  // the forward's tiles
    int32_t piece, pieces;   // columns per piece of the backward (a multiple of 256), and pieces
    size_t clear_bytes;
    int32_t dx_ntiles;
    int32_t slices, kb_slice;
    bool direct;
    size_t off_sid, off_sp, off_zt, off_ent, off_coef, off_part, off_dl, off_sums, total;
};

// Whether a piece's two gradients run in one grid. Together they save the rounds in which SMs wait for the
// last tiles, which counts with few rows; apart they keep to one set of operands at a time, which counts
// once the weights and their gradient pass the 129 MB L2 by far. The whole backward, together and apart: 64 x
// 2048 x 32000 (131 MB of weights) 85 and 88 us, 512 x 2048 x 32000 171 and 179 us, 300 x 1024 x 50257 105 and
// 113 us; 1024 x 2048 x 32000 286 and 287 us, 2039 x 2048 x 32000 528 and 521 us; 4096 x 4096 x 50257 (412 MB)
// 3.23 and 3.14 ms, 16 x 4096 x 131072 (1074 MB) 517 and 504 us.
bool gradients_together(int64_t T, int32_t cols, int32_t D) { return T <= 512 && 2ll * cols * D <= (192ll << 20); }

// Slices of dx's contraction: a grid of few tiles leaves SMs idle, and each slice costs a round of fp32
// sums. Times in K steps of one SM (0.35 us): the rounds of dx's tiles or, in a grid with dW's (dw_steps,
// where a tile's epilogue is worth some 3 steps), all tiles over all SMs, whichever is longer, and the
// sums' traffic at 6 TB/s.
int32_t pick_slices(int64_t tiles, int32_t kblocks, double dw_steps, double sum_bytes) {
    int32_t best = 1;
    double best_t = 1e30;
    const double all = (static_cast<double>(tiles) * kblocks + dw_steps) / kPlanSms;
    for (int32_t s = 1; s <= 64 && s <= kblocks; ++s) {
        const int32_t kb = (kblocks + s - 1) / s;
        if ((kblocks + kb - 1) / kb != s) continue;
        const double t = std::max(static_cast<double>(ceil_div(tiles * s, kPlanSms)) * kb, all) +
                         (s > 1 ? s * sum_bytes / (0.35 * 6e6) : 0.0);
        if (t < best_t) best_t = t, best = s;
    }
    return best;
}

// Columns of the forward's tiles: a grid whose last round is nearly empty is worse than one of narrower
// tiles (one row tile and 32000 columns: 143 tiles of 224 for the 152 SMs instead of 125 of 256), and
// each tile costs what some 32 columns do besides its own.
int32_t pick_columns(int64_t mtiles, int32_t V) {
    int32_t best = kBN2;
    int64_t best_cost = INT64_MAX;
    for (int32_t bn = kBN2; bn >= 32; bn -= 32) {
        const int64_t cost = ceil_div(mtiles * ceil_div(V, bn), kPlanSms) * (bn + 32);
        if (cost < best_cost) best_cost = cost, best = bn;
    }
    return best;
}

void make_plan(int64_t T, int32_t D, int32_t V, int32_t K, LmPlan* p) {
    p->mtiles = static_cast<int32_t>(ceil_div(T, kBM));
    p->ntiles = static_cast<int32_t>(ceil_div(V, kBN2));
    p->fwd_bn = pick_columns(p->mtiles, V);
    p->fwd_ntiles = static_cast<int32_t>(ceil_div(V, p->fwd_bn));
    int64_t piece = kPieceBytes / (2 * T) / kBN2 * kBN2;
    piece = std::max<int64_t>(piece, kMinPiece);
    piece = std::min<int64_t>(piece, static_cast<int64_t>(p->ntiles) * kBN2);
    const int64_t pieces = ceil_div(static_cast<int64_t>(p->ntiles) * kBN2, piece);
    piece = ceil_div(p->ntiles, pieces) * kBN2;  // pieces of equal size
    p->piece = static_cast<int32_t>(piece);
    p->dx_ntiles = static_cast<int32_t>(ceil_div(D, kBN2));
    const int32_t kblocks = p->piece / kBK;
    const double dw_tiles = static_cast<double>(p->piece / kBM) * p->dx_ntiles;
    const double dw_steps =
        gradients_together(T, p->piece, D) ? dw_tiles * (static_cast<double>(ceil_div(T, kBK)) + 3.0) : 0.0;
    p->slices = pick_slices(static_cast<int64_t>(p->mtiles) * p->dx_ntiles, kblocks, dw_steps, 8.0 * T * D);
    p->kb_slice = (kblocks + p->slices - 1) / p->slices;
    p->direct = p->slices == 1 && p->piece >= V;
    // the status word, then one tile counter per piece, all cleared by each call
    p->pieces = static_cast<int32_t>(pieces);
    p->clear_bytes = sizeof(uint32_t) * (kFirstTicket + p->pieces);
    size_t off = (p->clear_bytes + kRegionAlign - 1) / kRegionAlign * kRegionAlign;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + kRegionAlign - 1) / kRegionAlign * kRegionAlign;
        return at;
    };
    const size_t t = static_cast<size_t>(T), tk = t * K;
    p->off_sid = take(4 * tk);
    p->off_sp = take(4 * tk);
    p->off_zt = take(4 * tk);
    p->off_ent = take(4 * t);
    p->off_coef = take(4 * t);
    // the forward's partials and the backward's buffers are never alive at once
    const size_t shared = off;
    p->off_part = take(8 * t * p->fwd_ntiles);
    const size_t fwd_end = off;
    off = shared;
    p->off_dl = take(2 * t * p->piece);
    p->off_sums = off;
    if (!p->direct) p->off_sums = take(4 * t * D * p->slices);
    p->total = std::max(off, fwd_end);
}

bool sizes_ok(int64_t T, int32_t D, int32_t V, int32_t K) {
    if (T <= 0 || D <= 0 || V <= 0 || K <= 0 || K > kLmMaxK || D % 64 != 0) return false;
    if (T >= (int64_t{1} << 31) || V > (1 << 30)) return false;
    // tile indices are 32-bit (the forward's tiles have 32 columns at least, an eighth of the full ones)
    const int64_t mt = ceil_div(T, kBM), nt = ceil_div(V, kBN2), dt = ceil_div(D, kBN2);
    return 8 * mt * nt < (int64_t{1} << 31) && 64 * mt * dt + 2 * nt * dt < (int64_t{1} << 31);
}

template <typename P>
P* at(const LmProblem& p, size_t off) {
    return reinterpret_cast<P*>(p.ws + off);
}

// Row tiles walked together: their rows of x (or dl) should take about a quarter of the 129 MB L2.
int32_t row_group(int64_t row_bytes, int32_t mtiles) {
    const int64_t g = (32ll << 20) / (row_bytes * kBM);
    return static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(g, mtiles)));
}

// Rows of the A box. A single row tile loads only the rows there are: the rest of the stage keeps what it
// held, and the products' rows that come of it are not looked at (rows do not mix in a product).
uint32_t box_rows(int64_t T) { return static_cast<uint32_t>(T >= kBM ? kBM : ceil_div(T, 8) * 8); }

moe_status_t prepare_targets(const LmProblem& p, const LmPlan& pl, bool backward, cudaStream_t stream) {
    uint32_t* status = reinterpret_cast<uint32_t*>(p.ws);
    if (cudaMemsetAsync(status, 0, backward ? pl.clear_bytes : sizeof(uint32_t), stream) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (p.teacher_ids == nullptr) return MOE_OK;  // the grids take the labels as they are
    float* coef = backward ? at<float>(p, pl.off_coef) : nullptr;
    const cudaError_t e =
        launch_pdl(k_lm_teacher, dim3(static_cast<unsigned>(ceil_div(p.T, 4))), dim3(128), 0, stream, p.teacher_ids,
                   p.teacher_logits, p.T, p.K, p.V, 1.0f / p.temperature, p.temperature, p.dloss,
                   at<int32_t>(p, pl.off_sid), at<float>(p, pl.off_sp), at<float>(p, pl.off_ent), coef, status);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// 1 / temperature, and what the tensor cores' accumulation takes off. They cut the fp32 accumulator's low
// bits off after each 16 products, towards zero, so that a logit comes out too small, by this part of itself per
// such step (measured for D = 256 to 65536): normal rows 1.1e-8 to 2.1e-8, rows that lean towards the weight row
// 1.6e-8 to 1.8e-8, rows whose products are all positive 2.2e-8 to 9.6e-8. 2^-26 (1.5e-8) per step, which is
// about the least that dense rows lose, is given back. Relative error of the loss at D = 4096, before and
// after: rows that lean towards their target 1.2e-5 and 1.5e-6, normal rows 6.1e-7 and 2.5e-7, rows with two
// thirds of their weight in a few columns 7.4e-7 and 3.0e-7.
// Rows of few non-zero elements lose nothing and are off by the factor instead: by 5e-7 with 2 % of the elements,
// by D 2^-30 at most, a 64th of the bound D 2^-24 of a sum of D products in fp32. D counts up to kScaleMaxD only,
// the largest that was measured.
constexpr int32_t kScaleMaxD = 65536;
double logit_scale(int32_t D, float temperature) {
    return (1.0 + std::min(D, kScaleMaxD) * 0x1p-30) / static_cast<double>(temperature);
}

LmArgs common_args(const LmProblem& p, const LmPlan& pl) {
    LmArgs a{};
    a.T = p.T;
    a.D = p.D;
    a.V = p.V;
    a.K = p.K;
    a.bm = static_cast<int32_t>(box_rows(p.T));
    // cross entropy: labels as the caller gave them (one outside the vocabulary finds no tile of the
    // forward; the join and the backward tell ignored labels from wrong ones)
    a.sid = p.teacher_ids ? at<int32_t>(p, pl.off_sid) : p.targets;
    a.ignore_index = p.ignore_index;
    a.dloss = p.dloss;
    a.sp = p.teacher_ids ? at<float>(p, pl.off_sp) : nullptr;
    a.scale2 = static_cast<float>(logit_scale(p.D, p.temperature) * 1.4426950408889634);
    a.status = reinterpret_cast<uint32_t*>(p.ws);
    return a;
}

}  // namespace

size_t lm_workspace_bytes(int64_t T, int32_t D, int32_t V, int32_t K) {
    if (!sizes_ok(T, D, V, K)) return 0;
    LmPlan pl{};
    make_plan(T, D, V, K, &pl);
    return pl.total;
}

moe_status_t launch_lm_fwd(const LmProblem& p, cudaStream_t stream) {
    LmPlan pl{};
    make_plan(p.T, p.D, p.V, p.K, &pl);
    CUtensorMap tx, tw;
    if (!make_tmap(&tx, p.x, p.D, p.T, kBK, box_rows(p.T)) || !make_tmap(&tw, p.w, p.D, p.V, kBK, pl.fwd_bn)) return MOE_ERR_CUDA;
    moe_status_t st = prepare_targets(p, pl, false, stream);
    if (st != MOE_OK) return st;
    LmArgs a = common_args(p, pl);
    a.mtiles = pl.mtiles;
    a.ntiles = pl.fwd_ntiles;
    a.bn = pl.fwd_bn;
    a.kblocks = p.D / kBK;
    a.group = row_group(2ll * p.D, pl.mtiles);
    a.zt = at<float>(p, pl.off_zt);
    a.part = at<float2>(p, pl.off_part);
    st = launch_gemm<LmLse>(tx, tw, a, sm_count_grid(static_cast<int64_t>(pl.mtiles) * pl.fwd_ntiles, p.sm_count),
                            stream);
    if (st != MOE_OK) return st;
    return launch_pdl(k_lm_join, dim3(static_cast<unsigned>(ceil_div(p.T, 32))), dim3(32 * kJoinWarps), 0, stream,
                      static_cast<const float2*>(a.part), pl.fwd_ntiles, p.T, p.K, a.sid, a.sp,
                      static_cast<const float*>(a.zt), static_cast<const float*>(at<float>(p, pl.off_ent)),
                      p.temperature, static_cast<float>(logit_scale(p.D, p.temperature)), a.scale2, p.ignore_index, p.V,
                      p.loss, p.lse, a.status) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

moe_status_t launch_lm_bwd(const LmProblem& p, cudaStream_t stream) {
    LmPlan pl{};
    make_plan(p.T, p.D, p.V, p.K, &pl);
    __nv_bfloat16* dl = at<__nv_bfloat16>(p, pl.off_dl);
    float* sums = at<float>(p, pl.off_sums);
    CUtensorMap tx, tw;
    GemmMaps grads{};
    if (!make_tmap(&tx, p.x, p.D, p.T, kBK, box_rows(p.T)) || !make_tmap(&tw, p.w, p.D, p.V, kBK, kBN2) ||
        !make_tmap(&grads.m[0], dl, pl.piece, p.T, kBK, box_rows(p.T)) ||
        !make_tmap(&grads.m[1], p.w, p.D, p.V, 64, kBK) || !make_tmap(&grads.m[2], dl, pl.piece, p.T, 64, kBK) ||
        !make_tmap(&grads.m[3], p.x, p.D, p.T, 64, kBK))
        return MOE_ERR_CUDA;
    moe_status_t st = prepare_targets(p, pl, true, stream);
    if (st != MOE_OK) return st;
    int32_t slices_used = 0;
    for (int64_t at_v = 0; at_v < p.V; at_v += pl.piece) {
        const int32_t v0 = static_cast<int32_t>(at_v);
        const int32_t cols =
            static_cast<int32_t>(std::min<int64_t>(pl.piece, ceil_div(p.V - at_v, kBN2) * kBN2));
        LmArgs a = common_args(p, pl);
        a.v0 = v0;
        a.pitch = pl.piece;
        a.lse = p.lse_in;
        a.coef = at<float>(p, pl.off_coef);
        a.mtiles = pl.mtiles;
        a.ntiles = cols / kBN2;
        a.bn = kBN2;
        a.kblocks = p.D / kBK;
        a.group = row_group(2ll * p.D, pl.mtiles);
        a.out0 = dl;
        st = launch_gemm<LmDlogits>(tx, tw, a, sm_count_grid(static_cast<int64_t>(a.mtiles) * a.ntiles, p.sm_count),
                                    stream);
        if (st != MOE_OK) return st;
        LmArgs b = a;
        b.ntiles = pl.dx_ntiles;
        b.kblocks = cols / kBK;
        b.kb_slice = pl.kb_slice;
        b.group = row_group(2ll * pl.kb_slice * kBK, pl.mtiles);
        b.direct = pl.direct;
        b.accumulate = v0 > 0;
        b.out0 = static_cast<__nv_bfloat16*>(p.dx);
        b.fout = sums;
        // the first piece is a whole one and starts every slice's sums; a shorter last piece adds to fewer
        const int32_t slices = static_cast<int32_t>(ceil_div(b.kblocks, b.kb_slice));
        slices_used = std::max(slices_used, slices);
        b.dx_tiles = p.dx ? b.mtiles * b.ntiles * slices : 0;
        // dW: row blocks whose tiles fill a round of the SMs, so that whole rows are written at a time
        b.dw_mtiles = cols / kBM;
        b.dw_kblocks = static_cast<int32_t>(ceil_div(p.T, kBK));
        b.dw_group = std::max(1, std::min(kPlanSms / b.ntiles, b.dw_mtiles));
        b.dw_tiles = p.dw ? b.dw_mtiles * b.ntiles : 0;
        b.out1 = static_cast<__nv_bfloat16*>(p.dw);
        const int32_t dx_tiles = b.dx_tiles, dw_tiles = b.dw_tiles;
        if (dx_tiles > 0 && dw_tiles > 0 && gradients_together(p.T, cols, p.D)) {
            b.ticket = b.status + kFirstTicket + v0 / pl.piece;
            st = launch_gemm<LmGrads<true>>(grads, b, sm_count_grid(static_cast<int64_t>(dx_tiles) + dw_tiles, p.sm_count),
                                            stream);
            if (st != MOE_OK) return st;
            continue;
        }
        if (dx_tiles > 0) {
            b.dw_tiles = 0;
            if ((st = launch_gemm<LmGrads<false>>(grads, b, sm_count_grid(dx_tiles, p.sm_count), stream)) != MOE_OK)
                return st;
        }
        if (dw_tiles > 0) {
            b.dx_tiles = 0;
            b.dw_tiles = dw_tiles;
            if ((st = launch_gemm<LmGrads<false>>(grads, b, sm_count_grid(dw_tiles, p.sm_count), stream)) != MOE_OK)
                return st;
        }
    }
    if (p.dx && !pl.direct) {
        const int64_t n4 = p.T * p.D / 4;
        const int64_t grid = std::min<int64_t>(ceil_div(n4, 256), 16ll * p.sm_count);
        if (launch_pdl(k_lm_sum_slices, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream,
                       reinterpret_cast<const float4*>(sums), slices_used, n4, static_cast<uint2*>(p.dx)) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // namespace moe
