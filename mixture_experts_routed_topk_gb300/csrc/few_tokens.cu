// few_tokens.cu -- the routed-expert layer for 1 to 32 tokens, in two kernels.
//
//   out[t] = sum_k s[t,k] W2[e] (SiLU(Wg[e] x_t) * (Wu[e] x_t)),   e = ids[t,k]
//
// With a few tokens the layer is the stream of its experts' weights: 6 F D bytes for each distinct expert, and 2
// to 64 operations for each of them. So the weights are the M side of every product (16 rows of an mma.sync
// tile), an expert's tokens are its N side (eight columns a tile, one tile for most experts), and everything is
// arranged for the stream. tcgen05 tiles have 128 rows of weights or more, which is too coarse to share a layer of
// 8 experts out over 152 SMs, and their rate is not needed: at the memory's rate an SM gets 12 weights a clock.
//
// The weights are cut into pieces of 16 rows x 64 elements of K. Each warp takes every eighth piece of its block's
// rows and copies the next two to four of them, with the columns of eight tokens, into a ring in shared memory in just
// the 16-byte units that its lanes will read: each lane reads only what it copied itself, so the only order to keep is
// a lane's wait for its own copies, and no warp waits for another until a tile's sums meet. Measured on the way
// (1 token, D = 7168, F = 2048, 8 experts; the weights alone take 104 us at the copy rate): a loading warp with TMA
// boxes of 2 KB 152 us and a ring filled by TMA for each warp 189 us (issue of small boxes and the chain of barrier,
// products and refill), loads into three sets of registers 143 us, this 109 us
// (115 us since H has two parts).
//
//   k_few_gate_up   a tile is 8 gate rows and the same 8 up rows of one expert, over all of D:
//                   the warps' sums meet in shared memory, SiLU(g) u is written to H (in two bf16 parts)
//   k_few_down      a tile is up to 16 rows of the output, over all experts and all of F: each warp adds an
//                   expert's sums, scaled by the tokens' scores in fp32, to its own 16 rows x T in shared
//                   memory; the warps' sums meet at the end, and out is rounded once
//
// Both kernels first make the plan that the routing kernels make for the large forward: the distinct experts
// in ascending order, for each the mask of its tokens and its first row of H. Every block makes it anew from
// the ids (or chooses them from the router's logits), which is quicker than another launch. The second kernel
// may start while the first one runs, makes its plan and copies its first weights before it waits for H.
//
// A pair whose score is 0 is passed over: it costs no weights. All sums are fp32, in a fixed order.
//
// Measured (calls in a graph, other experts in each; in brackets the weights at the copy rate, then the large forward):
// 1 x 2048 x 1408, 6 of 64 experts 24 us (15.3; 53); 1 x 7168 x 2048, 8 experts 113 us (104; 173); 8 x 4096 x 1536,
// 8 of 64 236 us (232; 260); 16 x 7168 x 2048, 8 of 64 751 us (726; 727), 8 of 256 1371 us (1339; 1301);
// 32 x 4096 x 1536, 8 of 128 622 us (614; 618).
// The large forward takes some 20 us more for its launches, but streams a large layer up to 6 % quicker: the two meet at
// some 3 GB of weights, and this is the quicker one below for up to 12 tokens (11 layers, 1 to 32 tokens). With more
// tokens the columns cost more than the weights they meet: 24 x 2048 x 1408, 6 of 64 206 us (146; 178),
// 32 x 2048 x 1408, 4 of 8 75 us (20; 52), 32 x 7168 x 2048, 8 of 32 514 us (416; 439). There tiles of 128 rows are the
// better layout. Which call to make is the caller's choice.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "gemm_pipeline.cuh"
#include "ptx_sm103.cuh"
#include "serve_internal.cuh"
#include "train_internal.cuh"

namespace moe {
namespace {

constexpr int kFewRows = 16;                        // weight rows of a tile
constexpr int kFewK = 64;                           // elements of K in a piece
constexpr int kFewF = kFewRows / 2;                 // f values of a gate/up tile
constexpr int kUnit = 512;                          // bytes of a 16-byte unit of every lane

// How a launch is laid out: the most column tiles, and rings as deep as two blocks' shared memory holds. A piece in a
// ring has 2 KB of weights and 1 KB of columns, or 2 KB of H's two parts.
template <int kTiles_>
struct Shape {
    static constexpr int kTiles = kTiles_, kWarps = 8, kBlocks = 2;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kUpDepth = kTiles == 4 ? 3 : 4, kDownDepth = kTiles == 4 ? 2 : 3;
    static constexpr int kUpBytes = kUpDepth * 6 * kUnit, kDownBytes = kDownDepth * 8 * kUnit;
    static constexpr int kRing = kUpBytes > kDownBytes ? kUpBytes : kDownBytes;  // a warp's
};

struct FewArgs {
    const __nv_bfloat16* x;
    const __nv_bfloat16* w13;
    const __nv_bfloat16* w2;
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

// The plan in shared memory: U experts, the bits of their tokens, their first slots (rows of H), and each
// slot's token and score.
struct Plan {
    int32_t* expert;
    uint32_t* mask;
    int32_t* base;
    int32_t* token;
    float* score;
};
constexpr int kPlanBytesPerPair = 20;

// Shared memory: the warps' rings (in which the plan is made first), their sums, the plan.
template <class S>
struct FewSmem {
    static constexpr int kRing = S::kWarps * S::kRing;
    static constexpr int kSums = S::kWarps * S::kTiles * 512;
    static_assert(kRing >= 4 * kMaxExperts + 8 * kFewMaxPairs, "room to make the plan in");
    static_assert(S::kBlocks * (kRing + kSums + 4 * S::kWarps + kPlanBytesPerPair * 256 + 1024) <= 228 * 1024, "fits");
    static_assert(kRing + kSums + 4 * S::kWarps + kPlanBytesPerPair * kFewMaxPairs <= 227 * 1024, "fits");
    static size_t bytes(int pairs) {
        return kRing + kSums + sizeof(int32_t) * S::kWarps + static_cast<size_t>(pairs) * kPlanBytesPerPair;
    }
    uint8_t* ring;
    float* red;  // [kWarps][8 kTiles][16]: a warp's sums of 16 rows for each column or token
    int32_t* sums;
    Plan plan;
    __device__ FewSmem(uint8_t* p, int pairs) {
        ring = p;
        red = reinterpret_cast<float*>(p + kRing);
        sums = reinterpret_cast<int32_t*>(p + kRing + kSums);
        plan.expert = sums + S::kWarps;
        plan.mask = reinterpret_cast<uint32_t*>(plan.expert + pairs);
        plan.base = reinterpret_cast<int32_t*>(plan.mask + pairs);
        plan.token = plan.base + pairs;
        plan.score = reinterpret_cast<float*>(plan.token + pairs);
    }
};

// Reads of ids, scores and logits go to L2. The down kernel makes its plan before it waits (see there): by then their
// writer has completed and L2 has what it wrote, but an SM on which no block has waited since may hold older lines in L1.
__device__ __forceinline__ float from_l2(const float* p) { return __ldcg(p); }
__device__ __forceinline__ float from_l2(const __nv_bfloat16* p) {
    return __bfloat162float(__ushort_as_bfloat16(__ldcg(reinterpret_cast<const unsigned short*>(p))));
}
__device__ __forceinline__ int32_t from_l2(const int32_t* p) { return __ldcg(p); }

// One token's choice as the router makes it: the K largest logits, equal ones by the lowest id, and their
// scores. One warp; a round takes the largest key below the last one's, so nothing is marked as taken.
template <typename L>
__device__ void choose(const L* row, int32_t E, int32_t K, bool normalize, int lane, int32_t* ids, float* scores) {
    constexpr int kHeld = 8;  // keys of a lane that stay in registers: up to 256 experts
    uint32_t key[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) key[i] = 32 * i + lane < E ? order_key(from_l2(row + 32 * i + lane)) : 0u;
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
        for (int32_t e = 32 * kHeld + lane; e < E; e += 32) look(order_key(from_l2(row + e)), e);
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
        for (int32_t e = 32 * kHeld + lane; e < E; e += 32) part += expf(from_l2(row + e) - m);
        part = warp_sum(part);
    }
    const float inv = 1.0f / part;
    __syncwarp();
    for (int k = lane; k < K; k += 32) scores[k] = m == -INFINITY ? 0.0f : scores[k] * inv;
}

// The plan of up to 32 pairs, by one warp with a pair to each lane, which compares itself to the others twice.
// Returns the number of experts. scratch: 96 words.
__device__ int plan_in_warp(int32_t id, float score, bool live, int pairs, int K, int lane, int32_t* scratch,
                            const Plan& plan) {
    constexpr int32_t kNone = 0x7fffffff;
    float* scores = reinterpret_cast<float*>(scratch + 32);
    scratch[lane] = live ? id : -1;
    scores[lane] = score;
    __syncwarp();
    const int token = lane / K;
    uint32_t mask = 0u;                        // the expert's tokens
    bool first = live, first_of_token = live;  // nobody before names the expert, or names it for this token
    float sum = 0.0f;                          // of a token that names an expert twice, in order
    for (int p = 0, t = 0, k = 0; p < pairs; ++p) {
        if (scratch[p] == id) {
            mask |= 1u << t;
            if (p < lane) first = false;
            if (t == token) {
                sum += scores[p];
                if (p < lane) first_of_token = false;
            }
        }
        if (++k == K) k = 0, ++t;
    }
    __syncwarp();
    scratch[lane] = first ? id : kNone;
    scratch[32 + lane] = first_of_token ? id : kNone;
    __syncwarp();
    int before = 0, base = 0;  // experts with lower ids, and their slots
    for (int p = 0; p < pairs; ++p) {
        before += scratch[p] < id ? 1 : 0;
        base += scratch[32 + p] < id ? 1 : 0;
    }
    if (first) {
        plan.expert[before] = id;
        plan.mask[before] = mask;
        plan.base[before] = base;
    }
    if (first_of_token) {
        const int slot = base + __popc(mask & ((1u << token) - 1u));
        plan.token[slot] = token;
        plan.score[slot] = sum;
    }
    return __popc(__ballot_sync(0xffffffffu, first));
}

// Makes the plan; returns the number of experts. scratch: the rings, before anything is copied into them.
template <class S, bool kFirst>
__device__ int make_plan(const FewArgs& a, uint8_t* scratch, const Plan& plan, int32_t* sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pairs = a.T * a.K;
    uint32_t* table = reinterpret_cast<uint32_t*>(scratch);  // [E] the tokens of each expert
    int32_t* ids = reinterpret_cast<int32_t*>(table + a.E);  // [pairs]
    float* scores = reinterpret_cast<float*>(ids + pairs);
    auto given_score = [&](int p) {
        return a.scores_bf16 ? from_l2(static_cast<const __nv_bfloat16*>(a.scores) + p)
                             : from_l2(static_cast<const float*>(a.scores) + p);
    };
    const bool speaks = kFirst && blockIdx.x == 0;  // writes what the caller gets to see
    if (a.logits != nullptr) {
        for (int t = warp; t < a.T; t += S::kWarps) {
            const int64_t row = static_cast<int64_t>(t) * a.E;
            if (a.logits_bf16)
                choose(static_cast<const __nv_bfloat16*>(a.logits) + row, a.E, a.K, a.normalize, lane, ids + t * a.K,
                       scores + t * a.K);
            else
                choose(static_cast<const float*>(a.logits) + row, a.E, a.K, a.normalize, lane, ids + t * a.K,
                       scores + t * a.K);
        }
        if (a.T > 1) __syncthreads();
        else __syncwarp();
        if (speaks && (a.T > 1 || warp == 0))
            for (int p = a.T > 1 ? tid : lane; p < pairs; p += a.T > 1 ? S::kThreads : 32) {
                a.ids_out[p] = ids[p];
                a.scores_out[p] = scores[p];
            }
    }
    // A block's first weights wait for this. 6 pairs: 1.7 us by the whole block, 0.9 us by one warp.
    if (pairs <= 32) {
        if (warp == 0) {
            int32_t id = 0;
            float score = 0.0f;
            if (lane < pairs) {
                id = a.logits ? ids[lane] : from_l2(a.ids + lane);
                score = a.logits ? scores[lane] : given_score(lane);
            }
            const bool bad = static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.E);
            __syncwarp();
            const int experts = plan_in_warp(id, score, lane < pairs && !bad && score != 0.0f, pairs, a.K, lane,
                                             reinterpret_cast<int32_t*>(scratch), plan);
            const bool any_bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) {
                sums[0] = experts;
                if (speaks) *a.status = any_bad ? MOE_DEV_BAD_EXPERT_ID : 0u;
            }
        }
        __syncthreads();
        return sums[0];
    }
    for (int e = tid; e < a.E; e += S::kThreads) table[e] = 0u;
    if (a.logits == nullptr)
        for (int p = tid; p < pairs; p += S::kThreads) {
            ids[p] = from_l2(a.ids + p);
            scores[p] = given_score(p);
        }
    __syncthreads();
    int bad = 0;
    for (int p = tid; p < pairs; p += S::kThreads) {
        const uint32_t e = static_cast<uint32_t>(ids[p]);
        if (e >= static_cast<uint32_t>(a.E)) bad = 1;
        else if (scores[p] != 0.0f) atomicOr(&table[e], 1u << (p / a.K));
    }
    bad = __syncthreads_or(bad);
    if (speaks && tid == 0) *a.status = bad ? MOE_DEV_BAD_EXPERT_ID : 0u;
    // ascending experts; (experts, slots) are counted together, in the halves of a word
    int32_t run = 0;
    for (int e0 = 0; e0 < a.E; e0 += S::kThreads) {
        const uint32_t m = e0 + tid < a.E ? table[e0 + tid] : 0u;
        const int32_t own = m ? (1 << 16) + __popc(m) : 0;
        int32_t upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        int32_t before = run + upto - own;
#pragma unroll
        for (int w = 0; w < S::kWarps; ++w) {
            if (w < warp) before += sums[w];
            run += sums[w];
        }
        if (m) {
            plan.expert[before >> 16] = e0 + tid;
            plan.mask[before >> 16] = m;
            plan.base[before >> 16] = before & 0xffff;
        }
        __syncthreads();
    }
    const int experts = run >> 16;
    for (int u = warp; u < experts; u += S::kWarps) {  // a lane per token
        const uint32_t m = plan.mask[u];
        if ((m >> lane) & 1u) {
            float s = 0.0f;
            for (int k = 0; k < a.K; ++k)
                if (ids[lane * a.K + k] == plan.expert[u]) s += scores[lane * a.K + k];
            const int slot = plan.base[u] + __popc(m & ((1u << lane) - 1u));
            plan.token[slot] = lane;
            plan.score[slot] = s;
        }
    }
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

// A lane's part of 64 elements of K of one row: the 16-byte units lane % 4 and lane % 4 + 4. The products run
// over K in an order of their own (step s takes words s of those units), the same for weights and tokens, so both
// come in 16-byte loads, two of which take a row's 128 bytes whole.
struct Units {
    uint32_t lo[4], hi[4];

    __device__ void take(const uint8_t* lo_at, const uint8_t* hi_at) {
        *reinterpret_cast<uint4*>(lo) = *reinterpret_cast<const uint4*>(lo_at);
        *reinterpret_cast<uint4*>(hi) = *reinterpret_cast<const uint4*>(hi_at);
    }
    // x; H, which the kernel before wrote, from L2; or zeros
    __device__ void take_x(const __nv_bfloat16* p, bool there) {
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(lo) = there ? __ldg(reinterpret_cast<const uint4*>(p)) : none;
        *reinterpret_cast<uint4*>(hi) = there ? __ldg(reinterpret_cast<const uint4*>(p + 32)) : none;
    }
    __device__ void take_h(const __nv_bfloat16* p, bool there) {
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(lo) = there ? __ldcg(reinterpret_cast<const uint4*>(p)) : none;
        *reinterpret_cast<uint4*>(hi) = there ? __ldcg(reinterpret_cast<const uint4*>(p + 32)) : none;
    }
};

// The weights of a piece as a lane holds them: rows lane / 4 and lane / 4 + 8.
struct Weights {
    Units top, bottom;
};

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there = true) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// A lane's own ring of pieces in shared memory: what it copies there it alone reads, so a wait for its own copies
// is all the order there is to keep. Unit i of all lanes lies together, without bank conflicts: the weights', then
// those of the first column tile's parts (x has one, H two). The other tiles of an expert with more than eight tokens
// are loaded when they are needed: rings that hold them too have room for fewer pieces, and took 708 us against 642 for
// 32 x 4096 x 1536, 8 of 128 experts (with every token among four of 8 experts 65 against 74). Loading a tile's columns
// while the one before is multiplied made 16 x 7168 x 2048 slower (806 us against 765) and 32 tokens 1 to 6 % faster.
template <class S, int kParts, int kDepth>
struct Ring {
    static constexpr int kSlot = (4 + 2 * kParts) * kUnit;
    static_assert(kDepth * kSlot <= S::kRing, "fits");
    uint8_t* mine;  // this lane's first unit of place 0
    int at = 0;
    __device__ Ring(uint8_t* ring, int warp, int lane) : mine(ring + warp * S::kRing + 16 * lane) {}
    __device__ uint32_t place(int i) const { return smem_addr(mine + i * kSlot); }
    __device__ void get(Weights& w, Units (&column)[kParts]) const {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        const uint8_t* p = mine + at * kSlot;
        w.top.take(p, p + kUnit);
        w.bottom.take(p + 2 * kUnit, p + 3 * kUnit);
#pragma unroll
        for (int i = 0; i < kParts; ++i) column[i].take(p + (4 + 2 * i) * kUnit, p + (5 + 2 * i) * kUnit);
    }
    __device__ void next() { at = at + 1 == kDepth ? 0 : at + 1; }
};

// The sums of a warp: 16 rows x 8 columns a tile. A single tile has two chains of products, so that one does
// not wait for the other.
template <int kTiles>
struct Sums {
    static constexpr int kChains = kTiles == 1 ? 2 : 1;
    float c[kTiles][kChains][4];

    __device__ void clear() {
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int h = 0; h < kChains; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[j][h][i] = 0.0f;
    }
    // Value i of tile j: row lane / 4 + 8 (i / 2), column 8 j + 2 (lane % 4) + i % 2.
    __device__ float value(int j, int i) const { return kChains == 2 ? c[j][0][i] + c[j][kChains - 1][i] : c[j][0][i]; }

    __device__ void add(int j, const Weights& w, const Units& b) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            mma_16x8x16(c[j][s % kChains], w.top.lo[s], w.bottom.lo[s], w.top.hi[s], w.bottom.hi[s], b.lo[s], b.hi[s]);
    }
};

// The warps' sums of a row for a column, in warp order.
template <class S>
__device__ __forceinline__ float sum_of_warps(const float* red, int row, int column) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < S::kWarps; ++w) s += red[(w * 8 * S::kTiles + column) * 16 + row];
    return s;
}

// A warp's way through its block's rows of weights, `pieces` pieces to each: it takes the pieces w, w + kWarps, ...
// of all the rows strung together, so that the warps' shares are equal however many pieces a row has. A row's
// place (major, minor) goes on by `step` from row to row, and minor counts up to `limit`.
struct Walk {
    int p, row = 0, major, minor;
    __device__ Walk(int warp, int2 start, int pieces, int2 step, int limit)
        : p(warp), major(start.x), minor(start.y) {
        settle(pieces, step, limit);
    }
    // Moves on from past a row's end; true in a new row.
    __device__ bool settle(int pieces, int2 step, int limit) {
        if (p < pieces) return false;
        do {
            p -= pieces;
            ++row;
            major += step.x;
            minor += step.y;
            if (minor >= limit) minor -= limit, ++major;
        } while (p >= pieces);
        return true;
    }
};

template <class S>
__global__ void __launch_bounds__(S::kThreads, S::kBlocks) k_few_gate_up(const FewArgs a) {
    constexpr int kTiles = S::kTiles;
    extern __shared__ __align__(16) uint8_t raw[];
    FewSmem<S> sm(raw, a.T * a.K);
    const Plan& plan = sm.plan;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    const int experts = make_plan<S, true>(a, sm.ring, plan, sm.sums);
    const int per_expert = a.F / kFewF, tiles = experts * per_expert, pieces = a.D / kFewK;
    const int first = blockIdx.x, stride = gridDim.x;
    const int rows = first < tiles ? (tiles - 1 - first) / stride + 1 : 0;  // the block's tiles
    griddep_launch_dependents();
    // a tile's place: expert of the plan, tile of the expert
    const int2 start = make_int2(first / per_expert, first % per_expert);
    const int2 step = make_int2(stride / per_expert, stride % per_expert);
    // copies into the ring, as far ahead as it is deep
    Walk ahead(warp, start, pieces, step, per_expert);
    bool on = false;  // whether this lane has a column of the expert whose pieces are copied
    const __nv_bfloat16 *column = nullptr, *gate = nullptr;
    const int64_t up = static_cast<int64_t>(a.F) * a.D;
    auto aim = [&] {
        if (ahead.row < rows) {
            const int u = ahead.major;
            on = (lane >> 2) < __popc(plan.mask[u]);
            column = a.x + (on ? static_cast<int64_t>(plan.token[plan.base[u] + (lane >> 2)]) * a.D : 0) + 8 * (lane & 3);
            gate = a.w13 + (2 * static_cast<int64_t>(plan.expert[u]) * a.F + ahead.minor * kFewF + (lane >> 2)) * a.D + 8 * (lane & 3);
        }
    };
    auto load = [&](uint32_t to) {
        if (ahead.row < rows) {
            const int k = ahead.p * kFewK;
            copy16(to, gate + k);
            copy16(to + kUnit, gate + k + 32);
            copy16(to + 2 * kUnit, gate + up + k);
            copy16(to + 3 * kUnit, gate + up + k + 32);
            copy16(to + 4 * kUnit, column + k, on);
            copy16(to + 5 * kUnit, column + k + 32, on);
            ahead.p += S::kWarps;
            if (ahead.settle(pieces, step, per_expert)) aim();
        }
        copy_group();
    };
    Ring<S, 1, S::kUpDepth> ring(sm.ring, warp, lane);
    aim();
#pragma unroll 1
    for (int i = 0; i < S::kUpDepth; ++i) load(ring.place(i));
    Walk now(warp, start, pieces, step, per_expert);
    Sums<kTiles> acc;
    for (int row = 0; row < rows; ++row) {
        const int tile = first + row * stride, u = tile / per_expert;
        const int count = __popc(plan.mask[u]), base = plan.base[u];
        acc.clear();
        while (now.row == row) {
            Weights w;
            Units b[1];
            ring.get(w, b);
            acc.add(0, w, b[0]);
#pragma unroll
            for (int j = 1; j < kTiles; ++j) {
                if (8 * j >= count) break;
                const int col = 8 * j + (lane >> 2);
                const bool there = col < count;
                b[0].take_x(a.x + (there ? static_cast<int64_t>(plan.token[base + col]) * a.D : 0) + now.p * kFewK + 8 * (lane & 3), there);
                acc.add(j, w, b[0]);
            }
            load(ring.place(ring.at));
            ring.next();
            now.p += S::kWarps;
            now.settle(pieces, step, per_expert);
        }
        // the warps' sums meet
        if (row > 0) __syncthreads();  // the last tile's have been read
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sm.red[((warp * kTiles + j) * 8 + 2 * (lane & 3) + (i & 1)) * 16 + (lane >> 2) + 8 * (i >> 1)] = acc.value(j, i);
        __syncthreads();
        for (int o = threadIdx.x; o < kFewF * count; o += S::kThreads) {
            const int f = o & 7, col = o >> 3;
            const float g = sum_of_warps<S>(sm.red, f, col), v = sum_of_warps<S>(sm.red, f + 8, col);
            // H goes on in two bf16 parts, which together are good to 2^-17. Rounded to one, as the large forward's, it
            // made up half of the output's error (2.3e-3 against 1.6e-3 of rounding the output alone), and 5 % less time.
            const float h = g / (1.0f + __expf(-g)) * v;
            // From 0x1.ffp127 on bf16 rounds to infinity: the first part is cut off instead, so that a finite H stays
            // one; infinity has no second part (infinity less infinity is not a number).
            const __nv_bfloat16 part = fabsf(h) < 0x1.ffp127f ? __float2bfloat16_rn(h) : __float2bfloat16_rz(h);
            const float left = isinf(h) ? 0.0f : h - __bfloat162float(part);
            __nv_bfloat16* to = a.h + static_cast<int64_t>(base + col) * a.F + (tile - u * per_expert) * kFewF + f;
            to[0] = part;
            to[static_cast<int64_t>(a.T) * a.K * a.F] = __float2bfloat16_rn(left);
        }
    }
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, S::kBlocks) k_few_down(const FewArgs a) {
    constexpr int kTiles = S::kTiles;
    extern __shared__ __align__(16) uint8_t raw[];
    FewSmem<S> sm(raw, a.T * a.K);
    const Plan& plan = sm.plan;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Before griddep_wait(): what the call reads was written by kernels that had completed when the gate/up kernel passed
    // its own wait, and every block of it lets this one start only after that. The reads here, of ids, scores, logits and
    // the first weights, go to L2, where those kernels' writes are.
    const int experts = make_plan<S, false>(a, sm.ring, plan, sm.sums);
    const int tiles = (a.D + a.rows - 1) / a.rows, pieces = a.F / kFewK;
    const int first = blockIdx.x, stride = gridDim.x;
    const int mine = first < tiles ? (tiles - 1 - first) / stride + 1 : 0;  // the block's tiles
    const int rows = mine * experts;                                        // and their rows of each expert
    // a row's place: the block's tile, expert of the plan
    const int2 start = make_int2(0, 0), step = make_int2(0, 1);
    Walk ahead(warp, start, pieces, step, experts);
    bool on = false, has_top = false, has_bottom = false;
    const __nv_bfloat16 *column = nullptr, *down = nullptr;
    auto aim = [&] {
        if (ahead.row < rows) {
            const int u = ahead.minor, d = (first + ahead.major * stride) * a.rows;
            const int end = min(a.rows, a.D - d);
            on = (lane >> 2) < __popc(plan.mask[u]);
            column = a.h + static_cast<int64_t>(plan.base[u] + (on ? lane >> 2 : 0)) * a.F + 8 * (lane & 3);
            has_top = (lane >> 2) < end;
            has_bottom = (lane >> 2) + 8 < end;
            down = a.w2 + (static_cast<int64_t>(plan.expert[u]) * a.D + d + (has_top ? lane >> 2 : 0)) * a.F + 8 * (lane & 3);
        }
    };
    auto load_weights = [&](uint32_t to) {
        if (ahead.row >= rows) return;
        const __nv_bfloat16* p = down + ahead.p * kFewK;
        const __nv_bfloat16* q = has_bottom ? p + 8 * static_cast<int64_t>(a.F) : p;
        copy16(to, p, has_top);
        copy16(to + kUnit, p + 32, has_top);
        copy16(to + 2 * kUnit, q, has_bottom);
        copy16(to + 3 * kUnit, q + 32, has_bottom);
    };
    const int64_t second = static_cast<int64_t>(a.T) * a.K * a.F;  // from a first part of H to its second
    auto load_columns = [&](uint32_t to) {
        if (ahead.row < rows) {
            const __nv_bfloat16* p = column + ahead.p * kFewK;
            copy16(to + 4 * kUnit, p, on);
            copy16(to + 5 * kUnit, p + 32, on);
            copy16(to + 6 * kUnit, p + second, on);
            copy16(to + 7 * kUnit, p + second + 32, on);
        }
        copy_group();
    };
    auto move_on = [&] {
        ahead.p += S::kWarps;
        if (ahead.settle(pieces, step, experts)) aim();
    };
    Ring<S, 2, S::kDownDepth> ring(sm.ring, warp, lane);
    const Walk begin = ahead;
    aim();
#pragma unroll 1
    for (int i = 0; i < S::kDownDepth; ++i) {
        load_weights(ring.place(i));
        move_on();
    }
    griddep_wait();  // H
    griddep_launch_dependents();
    ahead = begin;
    aim();
#pragma unroll 1
    for (int i = 0; i < S::kDownDepth; ++i) {
        load_columns(ring.place(i));
        move_on();
    }
    Walk now(warp, start, pieces, step, experts);
    float* own = sm.red + warp * 128 * kTiles;  // [token][16]
    Sums<kTiles> acc;
    int row = 0;
    for (int tile = first; tile < tiles; tile += stride) {
#pragma unroll
        for (int i = 0; i < 4 * kTiles; ++i) own[32 * i + lane] = 0.0f;
        for (int u = 0; u < experts; ++u, ++row) {
            const int count = __popc(plan.mask[u]), base = plan.base[u];
            acc.clear();
            while (now.row == row) {
                Weights w;
                Units b[2];
                ring.get(w, b);
                acc.add(0, w, b[0]);
                acc.add(0, w, b[1]);
#pragma unroll
                for (int j = 1; j < kTiles; ++j) {
                    if (8 * j >= count) break;
                    const int col = 8 * j + (lane >> 2);
                    const bool there = col < count;
                    const __nv_bfloat16* p = a.h + static_cast<int64_t>(base + (there ? col : 0)) * a.F + now.p * kFewK + 8 * (lane & 3);
                    b[0].take_h(p, there);
                    b[1].take_h(p + second, there);
                    acc.add(j, w, b[0]);
                    acc.add(j, w, b[1]);
                }
                const uint32_t to = ring.place(ring.at);
                load_weights(to);
                load_columns(to);
                if (ahead.row < rows) move_on();
                ring.next();
                now.p += S::kWarps;
                now.settle(pieces, step, experts);
            }
            __syncwarp();  // a token's sums belong to another lane with another expert
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                if (j > 0 && 8 * j >= count) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = 8 * j + 2 * (lane & 3) + i;
                    if (col < count) {
                        float* t = own + plan.token[base + col] * 16 + (lane >> 2);
                        const float s = plan.score[base + col];
                        t[0] = fmaf(s, acc.value(j, i), t[0]);
                        t[8] = fmaf(s, acc.value(j, 2 + i), t[8]);
                    }
                }
            }
        }
        __syncthreads();
        for (int o = threadIdx.x; o < 128 * kTiles; o += S::kThreads) {
            const int r = o & 15, t = o >> 4, d = tile * a.rows + r;
            if (r < a.rows && d < a.D && t < a.T)
                a.out[static_cast<int64_t>(t) * a.D + d] = __float2bfloat16_rn(sum_of_warps<S>(sm.red, r, t));
        }
        __syncthreads();
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
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

template <class S>
moe_status_t run(FewArgs& a, int blocks, cudaStream_t stream) {
    if (allow_smem<&k_few_gate_up<S>>() != cudaSuccess || allow_smem<&k_few_down<S>>() != cudaSuccess)
        return MOE_ERR_CUDA;
    const int pairs = a.T * a.K;
    const size_t smem = FewSmem<S>::bytes(pairs);
    // Down tiles of equal height, as many as fill whole rounds of the SMs: D = 2048 makes 147 tiles of 14 rows for
    // 152 SMs, where tiles of 16 would leave 24 SMs without one.
    const int rounds = static_cast<int>(ceil_div(a.D, static_cast<int64_t>(kFewRows) * blocks));
    a.rows = static_cast<int>(ceil_div(a.D, static_cast<int64_t>(rounds) * blocks));
    const int64_t most = static_cast<int64_t>(std::min(pairs, a.E)) * (a.F / kFewF);
    const int down = (a.D + a.rows - 1) / a.rows;
    if (launch_pdl(k_few_gate_up<S>, dim3(sm_count_grid(most, blocks)), dim3(S::kThreads), smem, stream, a) !=
            cudaSuccess ||
        launch_pdl(k_few_down<S>, dim3(sm_count_grid(down, blocks)), dim3(S::kThreads), smem, stream, a) !=
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
    a.w13 = static_cast<const __nv_bfloat16*>(p.w13);
    a.w2 = static_cast<const __nv_bfloat16*>(p.w2);
    // Two blocks to an SM keep more loads in flight: 8 x 4096 x 1536, 64 experts 235 us, against 250 with one. One
    // to an SM where the down kernel has no more than one full tile for each (D <= 16 SMs): its tiles would be cut
    // in half for two, and with one block of each kernel on an SM the down kernel is there and has its first
    // weights before the gate/up kernel ends (1 x 2048 x 1408, 6 experts: 24.1 us, against 26.2 with two; 4 x 2048:
    // 65.7 and 71.2; all with H in one part).
    const int blocks = (p.D <= kFewRows * p.sm_count ? 1 : 2) * p.sm_count;
    if (p.T <= 8) return run<Shape<1>>(a, blocks, stream);
    if (p.T <= 16) return run<Shape<2>>(a, blocks, stream);
    return run<Shape<4>>(a, blocks, stream);
}

}  // namespace moe
