// few_tokens.cu -- the routed-expert layer for 1 to 32 tokens, in two kernels.
//
//   out[t] = sum_k s[t,k] W2[e] (SiLU(Wg[e] x_t) * (Wu[e] x_t)),   e = ids[t,k]
//
// With a few tokens the layer is the stream of its experts' weights: 6 F D bytes for each distinct expert,
// and 2 to 64 operations for each of them. So the weights are the M side of every product (16 rows of an
// mma.sync tile), the tokens are its N side (eight columns a tile, a token keeps its column with every
// expert), and everything is arranged for the stream: one warp keeps a ring of 16 KB stages filled by TMA,
// eight warps take one 64-element piece of K of each stage. tcgen05 tiles have 128 rows of weights or more,
// which is too coarse to share a layer of 8 experts out over 152 SMs, and their rate is not needed: at the
// memory's rate an SM gets 12 weights a clock, the mma.sync path takes 1024 per column tile.
//
//   k_few_gate_up   a tile is 8 gate rows and the same 8 up rows of one expert, over all of D:
//                   the warps' sums meet in shared memory, SiLU(g) u is written to H (bf16)
//   k_few_down      a tile is up to 16 rows of the output, over all experts and all of F: each expert's sums
//                   are scaled by the tokens' scores in fp32 and stay in registers; out is rounded once
//
// Both kernels first make the plan that the routing kernels make for the large forward: the distinct experts
// in ascending order, for each the mask of its tokens and its first row of H. Every block makes it anew from
// the ids (or chooses them from the router's logits), which is quicker than another launch. The second kernel
// is launched while the first one's last weights are on their way, and fills its ring with W2 before it waits
// for H; that is what the two rings of less than half an SM's shared memory are for.
//
// A pair whose score is 0 is passed over: it costs no weights. All sums are fp32, in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "gemm_pipeline.cuh"
#include "ptx_sm103.cuh"
#include "serve_internal.cuh"
#include "train_internal.cuh"

namespace moe {
namespace {

constexpr int kFewWarps = 8;                        // warps that compute; one more loads
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewRows = 16;                        // weight rows of a tile
constexpr int kFewK = 64;                           // elements of K in a piece: a 128-byte swizzled row
constexpr int kFewPiece = kFewRows * kFewK * 2;     // 2 KB
constexpr int kFewStage = kFewWarps * kFewPiece;    // a piece for each warp
constexpr int kFewF = kFewRows / 2;                 // f values of a gate/up tile

// Ring stages, for kTiles column tiles: two blocks (one of each kernel) share an SM's 228 KB.
template <int kTiles>
constexpr int kFewStages = kTiles == 4 ? 5 : 6;

struct FewArgs {
    const __nv_bfloat16* x;
    const int32_t* ids;
    const void* scores;
    const void* logits;
    int32_t* ids_out;
    float* scores_out;
    __nv_bfloat16* h;
    __nv_bfloat16* out;
    uint32_t* status;
    int32_t T, D, F, E, K;
    int32_t rows;  // of a down tile
    bool scores_bf16, logits_bf16, normalize;
};

// The plan in shared memory: U experts, the bits of their tokens, their first slots (rows of H), and the
// score of each slot. pairs: the arrays' capacity.
struct Plan {
    int32_t* expert;
    uint32_t* mask;
    int32_t* base;
    float* score;
};
constexpr int kPlanBytesPerPair = 16;

struct FewBars {
    uint64_t full[8], empty[8];
    int abort;
    int32_t sums[kFewWarps];
};

template <int kTiles>
constexpr size_t few_smem_bytes(int pairs) {
    return 1024 + kFewStages<kTiles> * kFewStage + kFewWarps * kTiles * 512 + sizeof(FewBars) +
           static_cast<size_t>(pairs) * kPlanBytesPerPair;
}

template <int kTiles>
struct FewSmem {
    uint8_t* ring;
    float* red;  // [kFewWarps][kTiles][16][8]
    FewBars* bars;
    Plan plan;
    __device__ FewSmem(uint8_t* base, int pairs) {
        ring = base + ((1024u - (smem_addr(base) & 1023u)) & 1023u);  // the swizzle counts from 1024-byte lines
        uint8_t* p = ring + kFewStages<kTiles> * kFewStage;
        red = reinterpret_cast<float*>(p);
        p += kFewWarps * kTiles * 512;
        bars = reinterpret_cast<FewBars*>(p);
        p += sizeof(FewBars);
        plan.expert = reinterpret_cast<int32_t*>(p);
        plan.mask = reinterpret_cast<uint32_t*>(plan.expert + pairs);
        plan.base = reinterpret_cast<int32_t*>(plan.mask + pairs);
        plan.score = reinterpret_cast<float*>(plan.base + pairs);
    }
};

// One token's choice as the router makes it: the K largest logits, equal ones by the lowest id, and their
// scores. One warp; a round takes the largest key below the last one's, so nothing is marked as taken.
template <typename L>
__device__ void choose(const L* row, int32_t E, int32_t K, bool normalize, int lane, int32_t* ids, float* scores) {
    constexpr int kHeld = 8;  // keys of a lane that stay in registers: up to 256 experts
    uint32_t key[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) key[i] = 32 * i + lane < E ? order_key(to_float(row[32 * i + lane])) : 0u;
    uint32_t last = 0xffffffffu;
    int32_t last_id = -1;
    float m = 0.0f, part = 0.0f;
    for (int k = 0; k < K; ++k) {
        uint32_t best = 0u;  // below every logit's key
        int32_t at = 0;
        auto look = [&](uint32_t v, int32_t e) {
            if (v > best && (v < last || (v == last && e > last_id))) best = v, at = e;
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i) look(key[i], 32 * i + lane);
        for (int32_t e = 32 * kHeld + lane; e < E; e += 32) look(order_key(to_float(row[e])), e);
        last = __reduce_max_sync(0xffffffffu, best);
        last_id = static_cast<int32_t>(
            __reduce_min_sync(0xffffffffu, best == last ? static_cast<uint32_t>(at) : 0xffffffffu));
        const float z = key_value(last);
        if (k == 0) m = z;
        const float e = expf(z - m);
        part += e;
        if (lane == 0) {
            ids[k] = last_id;
            scores[k] = e;
        }
    }
    if (!normalize) {
        part = 0.0f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (key[i] != 0u) part += expf(key_value(key[i]) - m);
        for (int32_t e = 32 * kHeld + lane; e < E; e += 32) part += expf(to_float(row[e]) - m);
        part = warp_sum(part);
    }
    const float inv = 1.0f / part;
    __syncwarp();
    for (int k = lane; k < K; k += 32) scores[k] = m == -INFINITY ? 0.0f : scores[k] * inv;
}

// Makes the plan; returns the number of experts. scratch: the ring, before anything is loaded into it.
template <bool kFirst>
__device__ int make_plan(const FewArgs& a, uint8_t* scratch, const Plan& plan, FewBars* bars) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pairs = a.T * a.K;
    uint32_t* table = reinterpret_cast<uint32_t*>(scratch);  // [E] the tokens of each expert
    int32_t* ids = reinterpret_cast<int32_t*>(table + a.E);  // [pairs]
    float* scores = reinterpret_cast<float*>(ids + pairs);
    for (int e = tid; e < a.E; e += kFewThreads) table[e] = 0u;
    if (a.logits != nullptr) {
        for (int t = warp; t < a.T; t += kFewWarps + 1) {
            const int64_t row = static_cast<int64_t>(t) * a.E;
            if (a.logits_bf16)
                choose(static_cast<const __nv_bfloat16*>(a.logits) + row, a.E, a.K, a.normalize, lane, ids + t * a.K,
                       scores + t * a.K);
            else
                choose(static_cast<const float*>(a.logits) + row, a.E, a.K, a.normalize, lane, ids + t * a.K,
                       scores + t * a.K);
        }
    } else {
        for (int p = tid; p < pairs; p += kFewThreads) {
            ids[p] = a.ids[p];
            scores[p] = a.scores_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.scores)[p])
                                      : static_cast<const float*>(a.scores)[p];
        }
    }
    __syncthreads();
    int bad = 0;
    for (int p = tid; p < pairs; p += kFewThreads) {
        const uint32_t e = static_cast<uint32_t>(ids[p]);
        if (e >= static_cast<uint32_t>(a.E)) bad = 1;
        else if (scores[p] != 0.0f) atomicOr(&table[e], 1u << (p / a.K));
        if (kFirst && blockIdx.x == 0 && a.logits != nullptr) {
            a.ids_out[p] = ids[p];
            a.scores_out[p] = scores[p];
        }
    }
    bad = __syncthreads_or(bad);
    if (kFirst && blockIdx.x == 0 && tid == 0) *a.status = bad ? MOE_DEV_BAD_EXPERT_ID : 0u;
    // ascending experts; (experts, slots) are counted together, in the halves of a word
    int32_t run = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32 * kFewWarps) {
        const uint32_t m = warp < kFewWarps && e0 + tid < a.E ? table[e0 + tid] : 0u;
        const int32_t own = m ? (1 << 16) + __popc(m) : 0;
        int32_t upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (warp < kFewWarps && lane == 31) bars->sums[warp] = upto;
        __syncthreads();
        int32_t before = run + upto - own;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            if (w < warp) before += bars->sums[w];
            run += bars->sums[w];
        }
        if (m) {
            plan.expert[before >> 16] = e0 + tid;
            plan.mask[before >> 16] = m;
            plan.base[before >> 16] = before & 0xffff;
        }
        __syncthreads();
    }
    const int experts = run >> 16;
    for (int u = warp; u < experts; u += kFewWarps + 1) {  // a lane per token
        const uint32_t m = plan.mask[u];
        if ((m >> lane) & 1u) {
            float s = 0.0f;
            for (int k = 0; k < a.K; ++k)
                if (ids[lane * a.K + k] == plan.expert[u]) s += scores[lane * a.K + k];
            plan.score[plan.base[u] + __popc(m & ((1u << lane) - 1u))] = s;
        }
    }
    // the ring's next writer is TMA
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    return experts;
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// This lane's part of a column tile's 64 elements of K: the 16-byte units lane % 4 and lane % 4 + 4 of the
// row of column lane / 4. The products run over K in an order of their own (step s takes words s of those
// units), the same for weights and tokens, so both come in 16-byte loads.
struct Column {
    uint4 lo, hi;
};

template <int kTiles>
__device__ __forceinline__ void multiply(float (&acc)[kTiles][4], const uint8_t* piece, const Column (&b)[kTiles],
                                         uint32_t mask, int lane) {
    const int row = lane >> 2;
    const uint8_t* p = piece + row * 128 + (((lane & 3) ^ row) << 4);  // rows 0-7 and 8-15 have the same swizzle
    const uint8_t* q = piece + row * 128 + (((lane & 3) ^ row ^ 4) << 4);
    uint32_t a0[4], a1[4], a2[4], a3[4];
    *reinterpret_cast<uint4*>(a0) = *reinterpret_cast<const uint4*>(p);
    *reinterpret_cast<uint4*>(a1) = *reinterpret_cast<const uint4*>(p + 1024);
    *reinterpret_cast<uint4*>(a2) = *reinterpret_cast<const uint4*>(q);
    *reinterpret_cast<uint4*>(a3) = *reinterpret_cast<const uint4*>(q + 1024);
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
        if (kTiles > 1 && ((mask >> (8 * j)) & 0xffu) == 0u) continue;  // none of the tile's tokens
        const uint32_t lo[4] = {b[j].lo.x, b[j].lo.y, b[j].lo.z, b[j].lo.w};
        const uint32_t hi[4] = {b[j].hi.x, b[j].hi.y, b[j].hi.z, b[j].hi.w};
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_16x8x16(acc[j], a0[s], a1[s], a2[s], a3[s], lo[s], hi[s]);
    }
}

// Adds up the warps' 16 x 8 tiles: every warp stores its own, then sum(row, token) adds them in warp order.
template <int kTiles>
struct WarpTiles {
    float* red;
    __device__ void store(const float (&acc)[kTiles][4], int warp, int lane) {
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory");  // the last tile has been read
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            float* p = red + (warp * kTiles + j) * 128 + (lane >> 2) * 8 + (lane & 3) * 2;
            *reinterpret_cast<float2*>(p) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2*>(p + 64) = make_float2(acc[j][2], acc[j][3]);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory");
    }
    __device__ float sum(int row, int token) const {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) s += red[(w * kTiles + token / 8) * 128 + row * 8 + token % 8];
        return s;
    }
};

// A place in a ring of kStages.
template <int kStages>
struct RingAt {
    uint32_t s = 0, phase = 0;
    __device__ void next() {
        if (++s == kStages) s = 0, phase ^= 1u;
    }
};

template <int kTiles>
__device__ void setup(FewBars* bars, const CUtensorMap* map) {
    if (threadIdx.x == 0) {
        bars->abort = 0;
        for (int s = 0; s < kFewStages<kTiles>; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], kFewWarps);
        }
        mbar_init_fence();
        tma_prefetch_descriptor(map);
    }
}

// The loading warp's part of a stage: once the stage is empty, n pieces of `bytes` each, lane i issuing
// load(i, destination). False when the wait gave up.
template <int kTiles, class Load>
__device__ __forceinline__ bool fill(RingAt<kFewStages<kTiles>>& at, uint8_t* ring, FewBars* bars, uint32_t* status,
                                     int n, uint32_t bytes, int lane, Load load) {
    int ok = 1;
    if (lane == 0) {
        ok = mbar_wait(&bars->empty[at.s], at.phase ^ 1u, &bars->abort, status, MOE_DEV_TIMEOUT) ? 1 : 0;
        if (ok) mbar_arrive_expect_tx(&bars->full[at.s], n * bytes);
    }
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    if (lane < n) load(lane, ring + at.s * kFewStage + lane * kFewPiece, &bars->full[at.s]);
    at.next();
    return true;
}

// After a wait that gave up: the copies in flight get a moment to land before the block's memory is freed.
template <int kTiles>
__device__ void land(RingAt<kFewStages<kTiles>> at, uint32_t filled, FewBars* bars) {
    constexpr uint32_t kStages = kFewStages<kTiles>;
    const unsigned long long t0 = global_timer_ns();
    for (uint32_t i = 0; i < kStages && i < filled; ++i) {
        at.phase ^= at.s == 0 ? 1u : 0u;
        at.s = at.s == 0 ? kStages - 1 : at.s - 1;
        while (!mbar_try_wait(&bars->full[at.s], at.phase) && global_timer_ns() - t0 < 2000000ull) {
        }
    }
}

template <int kTiles>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_few_gate_up(const __grid_constant__ CUtensorMap w13, const FewArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    FewSmem<kTiles> sm(raw, a.T * a.K);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    setup<kTiles>(sm.bars, &w13);
    griddep_wait();
    const int experts = make_plan<true>(a, sm.ring, sm.plan, sm.bars);
    const int per_expert = a.F / kFewF, tiles = experts * per_expert, pieces = a.D / kFewK;
    RingAt<kFewStages<kTiles>> at;
    if (warp == kFewWarps) {
        bool ok = true;
        uint32_t filled = 0;
        for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
            const int u = tile / per_expert, f = (tile - u * per_expert) * kFewF, e = sm.plan.expert[u];
            for (int c = 0; ok && c < pieces; c += kFewWarps, ++filled)
                ok = fill<kTiles>(at, sm.ring, sm.bars, a.status, min(kFewWarps, pieces - c), kFewPiece, lane,
                                  [&](int i, uint8_t* to, uint64_t* bar) {
                                      tma_load_3d(to, &w13, bar, (c + i) * kFewK, f, 2 * e);
                                  });
        }
        // the last loads are on their way: the down kernel may start on its own
        griddep_launch_dependents();
        if (!ok && lane == 0) land<kTiles>(at, filled, sm.bars);
        return;
    }
    auto columns = [&](int tile, int c, Column (&b)[kTiles]) {
        const uint32_t mask = tile < tiles && c + warp < pieces ? sm.plan.mask[tile / per_expert] : 0u;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            const int t = 8 * j + (lane >> 2);
            b[j].lo = b[j].hi = make_uint4(0u, 0u, 0u, 0u);
            if ((mask >> t) & 1u) {
                const __nv_bfloat16* p = a.x + static_cast<int64_t>(t) * a.D + (c + warp) * kFewK + 8 * (lane & 3);
                b[j].lo = __ldg(reinterpret_cast<const uint4*>(p));
                b[j].hi = __ldg(reinterpret_cast<const uint4*>(p + 32));
            }
        }
    };
    WarpTiles<kTiles> meet{sm.red};
    Column next[kTiles];
    columns(blockIdx.x, 0, next);
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int u = tile / per_expert;
        const uint32_t mask = sm.plan.mask[u];
        float acc[kTiles][4] = {};
        for (int c = 0; c < pieces; c += kFewWarps) {
            Column b[kTiles];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) b[j] = next[j];
            // a stage ahead, over the end of the tile
            if (c + kFewWarps < pieces) columns(tile, c + kFewWarps, next);
            else columns(tile + gridDim.x, 0, next);
            mbar_wait(&sm.bars->full[at.s], at.phase, &sm.bars->abort, a.status, MOE_DEV_TIMEOUT);
            if (c + warp < pieces)
                multiply<kTiles>(acc, sm.ring + at.s * kFewStage + warp * kFewPiece, b, mask, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.bars->empty[at.s]);
            at.next();
        }
        meet.store(acc, warp, lane);
        const int f = threadIdx.x & 7, t = threadIdx.x >> 3;
        if (t < 8 * kTiles && ((mask >> t) & 1u)) {
            const float g = meet.sum(f, t), up = meet.sum(f + 8, t);
            const int64_t slot = sm.plan.base[u] + __popc(mask & ((1u << t) - 1u));
            // H is rounded to bf16 here, as the large forward's
            a.h[slot * a.F + (tile - u * per_expert) * kFewF + f] = __float2bfloat16_rn(g / (1.0f + __expf(-g)) * up);
        }
    }
}

template <int kTiles>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_few_down(const __grid_constant__ CUtensorMap w2, const FewArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    FewSmem<kTiles> sm(raw, a.T * a.K);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    setup<kTiles>(sm.bars, &w2);
    // Before griddep_wait(): ids, scores and logits were written by kernels that had completed when the gate/up
    // kernel passed its own wait, and it lets this one start only after that; nobody writes the weights.
    const int experts = make_plan<false>(a, sm.ring, sm.plan, sm.bars);
    const int tiles = (a.D + a.rows - 1) / a.rows, pieces = a.F / kFewK;
    RingAt<kFewStages<kTiles>> at;
    if (warp == kFewWarps) {
        bool ok = true;
        uint32_t filled = 0;
        for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x)
            for (int u = 0; ok && u < experts; ++u) {
                const int row = sm.plan.expert[u] * a.D + tile * a.rows;
                for (int c = 0; ok && c < pieces; c += kFewWarps, ++filled)
                    ok = fill<kTiles>(at, sm.ring, sm.bars, a.status, min(kFewWarps, pieces - c),
                                      a.rows * kFewK * 2, lane, [&](int i, uint8_t* to, uint64_t* bar) {
                                          tma_load_2d(to, &w2, bar, (c + i) * kFewK, row);
                                      });
            }
        griddep_launch_dependents();
        griddep_wait();
        if (!ok && lane == 0) land<kTiles>(at, filled, sm.bars);
        return;
    }
    griddep_wait();  // H
    auto columns = [&](int u, int c, Column (&b)[kTiles]) {
        const bool live = u < experts && c + warp < pieces;
        const uint32_t mask = live ? sm.plan.mask[u] : 0u;
        const int64_t base = live ? sm.plan.base[u] : 0;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            const int t = 8 * j + (lane >> 2);
            b[j].lo = b[j].hi = make_uint4(0u, 0u, 0u, 0u);
            if ((mask >> t) & 1u) {
                const __nv_bfloat16* p =
                    a.h + (base + __popc(mask & ((1u << t) - 1u))) * a.F + (c + warp) * kFewK + 8 * (lane & 3);
                b[j].lo = __ldcg(reinterpret_cast<const uint4*>(p));
                b[j].hi = __ldcg(reinterpret_cast<const uint4*>(p + 32));
            }
        }
    };
    WarpTiles<kTiles> meet{sm.red};
    Column next[kTiles];
    columns(0, 0, next);
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        float total[kTiles][4] = {};
        for (int u = 0; u < experts; ++u) {
            const uint32_t mask = sm.plan.mask[u];
            float acc[kTiles][4] = {};
            for (int c = 0; c < pieces; c += kFewWarps) {
                Column b[kTiles];
#pragma unroll
                for (int j = 0; j < kTiles; ++j) b[j] = next[j];
                if (c + kFewWarps < pieces) columns(u, c + kFewWarps, next);
                else columns(u + 1 < experts ? u + 1 : 0, 0, next);  // the next expert, or the next tile's first
                mbar_wait(&sm.bars->full[at.s], at.phase, &sm.bars->abort, a.status, MOE_DEV_TIMEOUT);
                if (c + warp < pieces)
                    multiply<kTiles>(acc, sm.ring + at.s * kFewStage + warp * kFewPiece, b, mask, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.bars->empty[at.s]);
                at.next();
            }
            // only tokens of this expert: another's column is 0 times weights that need not be finite
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = 8 * j + 2 * (lane & 3) + i;
                    if ((mask >> t) & 1u) {
                        const float s = sm.plan.score[sm.plan.base[u] + __popc(mask & ((1u << t) - 1u))];
                        total[j][i] = fmaf(s, acc[j][i], total[j][i]);
                        total[j][2 + i] = fmaf(s, acc[j][2 + i], total[j][2 + i]);
                    }
                }
        }
        meet.store(total, warp, lane);
        for (int o = threadIdx.x; o < 128 * kTiles; o += 32 * kFewWarps) {
            const int r = o & 15, t = o >> 4, d = tile * a.rows + r;
            if (r < a.rows && d < a.D && t < a.T)
                a.out[static_cast<int64_t>(t) * a.D + d] = __float2bfloat16_rn(meet.sum(r, t));
        }
    }
}

template <auto kKernel>
cudaError_t allow_smem() {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

template <int kTiles>
moe_status_t run(const CUtensorMap& w13, const CUtensorMap& w2, const FewArgs& a, int sm_count, cudaStream_t stream) {
    if (allow_smem<&k_few_gate_up<kTiles>>() != cudaSuccess || allow_smem<&k_few_down<kTiles>>() != cudaSuccess)
        return MOE_ERR_CUDA;
    const int pairs = a.T * a.K;
    const size_t smem = few_smem_bytes<kTiles>(pairs);
    const int64_t most = static_cast<int64_t>(std::min(pairs, a.E)) * (a.F / kFewF);
    const int down = (a.D + a.rows - 1) / a.rows;
    if (launch_pdl(k_few_gate_up<kTiles>, dim3(sm_count_grid(most, sm_count)), dim3(kFewThreads), smem, stream, w13, a) !=
            cudaSuccess ||
        launch_pdl(k_few_down<kTiles>, dim3(sm_count_grid(down, sm_count)), dim3(kFewThreads), smem, stream, w2, a) !=
            cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

}  // namespace

moe_status_t launch_few(const FewProblem& p, cudaStream_t stream) {
    FewArgs a{};
    a.x = static_cast<const __nv_bfloat16*>(p.x);
    a.ids = p.ids;
    a.scores = p.scores;
    a.scores_bf16 = p.scores_dtype == MOE_SCORES_BF16;
    a.logits = p.logits;
    a.logits_bf16 = p.logits_dtype == MOE_DTYPE_BF16;
    a.normalize = p.normalize;
    a.ids_out = p.ids_out;
    a.scores_out = p.scores_out;
    a.h = static_cast<__nv_bfloat16*>(p.h);
    a.out = static_cast<__nv_bfloat16*>(p.out);
    a.status = p.status;
    a.T = p.T;
    a.D = p.D;
    a.F = p.F;
    a.E = p.E;
    a.K = p.K;
    // Down tiles of equal height, as many as fill whole rounds of the SMs: D = 2048 makes 147 tiles of 14 rows for
    // 152 SMs, where tiles of 16 would leave 24 SMs without one.
    const int rounds = static_cast<int>(ceil_div(p.D, static_cast<int64_t>(kFewRows) * p.sm_count));
    a.rows = static_cast<int>(ceil_div(p.D, static_cast<int64_t>(rounds) * p.sm_count));
    CUtensorMap w13, w2;
    if (!make_tmap_pairs(&w13, p.w13, static_cast<uint64_t>(p.D), static_cast<uint64_t>(p.F),
                         static_cast<uint64_t>(p.E) * 2, kFewK, kFewF) ||
        !make_tmap(&w2, p.w2, static_cast<uint64_t>(p.F), static_cast<uint64_t>(p.E) * p.D, kFewK,
                   static_cast<uint32_t>(a.rows)))
        return MOE_ERR_CUDA;
    if (p.T <= 8) return run<1>(w13, w2, a, p.sm_count, stream);
    if (p.T <= 16) return run<2>(w13, w2, a, p.sm_count, stream);
    return run<4>(w13, w2, a, p.sm_count, stream);
}

}  // namespace moe
