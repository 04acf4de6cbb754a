// sample.cu -- the choice of the next token of each row of logits, from a given uniform number.
//
//   order      tokens by logit, largest first, equal ones by the lowest number
//   kept       the first top_k of them; of these the shortest run whose share of the probabilities
//              softmax(z / temperature) of those top_k reaches top_p; of these the ones with at least min_p times the
//              largest probability: always a run from the start of the order, cut at one (logit, number)
//   token      the first, by number, whose running sum of kept probabilities exceeds u times their sum
//
// Where many small probabilities are added up, two ways of adding disagree about which token a number falls to. So
// a weight exp((z - max) / temperature) is an integer in units of 2^-44, of which each loses less than one, made
// from a logarithm in two floats, a table of 2^(j/256) and a cubic, to 2^-30 of itself (the floats' roundings add up to
// 8.4e-10; 4.5e-10 is the most that a million random logits showed); sums of them are exact and in any order the same,
// and cuts and choice are integer comparisons. A row gives the same token whatever the grid, and the one that 64-bit
// arithmetic gives but for numbers within 2^-30 + V 2^-44 of a border. From V = 2^19 on, where sums could pass 63 bits, a
// pass of its own finds the finest unit, down to 2^-61, in which the row's own sum stays below 2^62: all tokens together
// then lose V 2^-60 of it at most. (Taken from 2^18 on, that pass made 64 x 262144 bf16 without a filter 109 us from 56.)
//
// A row is shared by a cluster of one to eight blocks, each of which owns a run of it. Filters need one histogram of
// the row: 16 bins to each halving of the weight, with counts and weights, merged over the cluster. The cut lies in
// one bin; its tokens (some hundreds) go to the first block, which sorts them. Bins with more tokens than the
// list holds are split again by the logits' bits, down to a single logit, whose ties are cut by number. Bound by
// latency for a few rows, by instruction issue for many: a pass over the weights has some 75 instructions for a warp's 32
// tokens, one that only looks for the largest logit about 4. A row without a filter passes four cluster barriers, one with
// top-k seven; they are the smaller part of a row's time (0.24 us each in a kernel of nothing else, of 512 threads and one to
// eight blocks), the rest is the passes' own latency and the sorts.
//
// Measured (calls in a graph): 1 x 32000 f32 without a filter 10 us, with top-k 17, top-p 22, both 17, min-p 11;
// 64 x 131072 bf16 33, 25, 96, 25 and 23 us; 256 x 131072 f32 with top-p 274 us, where reading the logits once takes
// 20. Of the 96 us the histogram takes 24, the list 10 and its sort 13, the last sums 18. Tried without gain: weights
// without branches and conversions, a histogram without counts; an estimate of the cut from every eighth token, with
// finer bins around it, took 136 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "exp2_table.cuh"
#include "ptx_sm103.cuh"
#include "serve_internal.cuh"
#include "train_internal.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kList = 2048;  // tokens of a bin that are sorted
constexpr int kPerOctave = 16;

struct SampleArgs {
    const float *uniform, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    int32_t* token;
    float* logprob;
    int32_t V;
    int shift;  // weights are in units of 2^-shift, or of finer ones from kWideV on
};
constexpr int kShift = 44;
constexpr int32_t kWideV = 1 << (63 - kShift);  // fewer of the largest weight stay below 2^63

struct Histogram {
    uint32_t count[kBins], lo[kBins], hi[kBins];
};
struct Totals {
    uint64_t weight[kBins];
    uint32_t count[kBins];
};
// Where a cut lies: kept are the tokens of larger keys, and of this key those up to this number.
struct Cut {
    uint32_t key;
    int32_t last;
};

struct SampleSmem {
    uint64_t table[256];
    Histogram hist;
    Totals merged;     // this block's share of the cluster's histogram
    Totals first;      // the whole cluster's, by weight
    Totals split;      // of one bin, by key
    uint64_t list[kList];
    uint64_t runs[kWarps][32];  // a warp's sums over its runs of steps
    uint64_t sums[kWarps];
    uint32_t counts[kWarps];
    uint32_t listed;
    uint32_t best;     // this block's largest
    uint64_t total;    // this block's kept weight
    Cut cut;           // the first block's answer
    uint64_t cut_weight;
    int32_t found_bin;
    uint32_t before_count;
    uint64_t before_weight;
    int32_t chosen;    // the block's answer in a search by number, or -1
    float c_hi, c_lo;  // 256 log2(e) / temperature
    uint64_t share;    // top_p in units of 2^-64
    uint32_t least;    // the smallest key that min_p keeps
};

// The largest of a piece's elements; not a number where one of them is none.
__device__ __forceinline__ float larger(float a, float b) {
    float v;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
    return v;
}
template <typename T>
__device__ __forceinline__ float largest_of(const uint4& piece);
template <>
__device__ __forceinline__ float largest_of<float>(const uint4& p) {
    return larger(larger(__uint_as_float(p.x), __uint_as_float(p.y)), larger(__uint_as_float(p.z), __uint_as_float(p.w)));
}
template <>
__device__ __forceinline__ float largest_of<__nv_bfloat16>(const uint4& p) {
    const auto* v = reinterpret_cast<const __nv_bfloat162*>(&p);
    const float2 m = __bfloat1622float2(__hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3])));
    return larger(m.x, m.y);
}
template <>
__device__ __forceinline__ float largest_of<__half>(const uint4& p) {
    const auto* v = reinterpret_cast<const __half2*>(&p);
    const float2 m = __half22float2(__hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3])));
    return larger(m.x, m.y);
}

template <typename T>
struct Row {
    static constexpr int kC = 16 / static_cast<int>(sizeof(T));
    static constexpr int kStep = 32 * kC;  // tokens that a warp takes at once
    const T* z;
    int32_t V;
    int lead;               // elements of the first 16-byte piece that come before the row
    int32_t begin, end;     // this warp's steps
    int32_t run;            // steps in a run, of which a warp has up to 32

    __device__ int32_t number(int32_t step, int lane) const { return (step * 32 + lane) * kC - lead; }
    // Whether all lanes' pieces of the step are the row's.
    __device__ bool inside(int32_t step) const { return step * kStep >= lead && (step + 1) * kStep - lead <= V; }
    __device__ static void keys_of(const uint4& piece, uint32_t (&key)[kC]) {
        T v[kC];
        *reinterpret_cast<uint4*>(v) = piece;
#pragma unroll
        for (int e = 0; e < kC; ++e) key[e] = order_key(to_float(v[e]));
    }
    // The keys of a lane's tokens in a step, in order of their numbers; 0 for none. Returns the first one's number.
    __device__ int32_t load(int32_t step, int lane, uint32_t (&key)[kC]) const {
        const int32_t j = number(step, lane);
        if (j >= 0 && j + kC <= V) {
            keys_of(__ldg(reinterpret_cast<const uint4*>(z + j)), key);
        } else {
#pragma unroll
            for (int e = 0; e < kC; ++e) key[e] = j + e >= 0 && j + e < V ? order_key(to_float(z[j + e])) : 0u;
        }
        return j;
    }
};

// A weight from a logit, the row's largest and 256 log2(e) / temperature in two floats.
struct Weigh {
    const uint64_t* table;
    float max, c_hi, c_lo;
    int shift;

    // 256 log2 of the weight; the part that a float does not hold in `rest`.
    __device__ float exponent(float z, float* rest) const {
        const float d = z - max, b = z - d;
        const float lost = (z - (d + b)) + (b - max);  // z - max is d + lost
        // a rounded product, whose error goes to the rest: contracted into what p is used in, it would count twice (up to
        // 3e-6 of the weight)
        const float p = __fmul_rn(d, c_hi);
        *rest = fmaf(d, c_lo, fmaf(lost, c_hi, fmaf(d, c_hi, -p)));
        return p;
    }
    __device__ uint64_t operator()(float z) const {
        if (z == max) return uint64_t{1} << shift;  // also where both are infinite
        float rest;
        const float p = exponent(z, &rest);
        if (!(p > -256.0f * (shift + 1))) return 0u;
        const int k = __float2int_rd(p);
        const float x = ((p - static_cast<float>(k)) + rest) * (0.69314718056f / 256.0f);
        const float f = x * fmaf(x, fmaf(x, 1.0f / 6.0f, 0.5f), 1.0f);  // 2^(..) - 1
        const uint64_t t = table[k & 255];
        const int64_t add = static_cast<int64_t>(__float2int_rn(f * 4294967296.0f)) * static_cast<int64_t>(t >> 32);
        const int by = 62 - shift - (k >> 8);
        return by > 63 ? 0u : (t + static_cast<uint64_t>(add)) >> by;
    }
    // Bins go down by weight; the last holds all that is left.
    __device__ int bin(float z) const {
        if (z == max) return 0;
        const float t = (z - max) * c_hi * (-kPerOctave / 256.0f);
        return t < kBins - 1 ? static_cast<int>(t) : kBins - 1;
    }
};

__device__ __forceinline__ uint64_t warp_upto(uint64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

__device__ __forceinline__ uint64_t warp_total(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The least weight, 1 or more, that is a share (in units of 2^-64) of a sum.
__device__ __forceinline__ uint64_t share_of(uint64_t share, uint64_t sum) {
    const uint64_t need = __umul64hi(share, sum) + (share * sum != 0u ? 1u : 0u);
    return need > 0u ? need : 1u;
}

template <typename T>
struct Sampler {
    SampleSmem& sm;
    cg::cluster_group cluster;
    Row<T> row;
    Weigh weigh;
    int rank, ranks, lane, warp, tid;

    // piece_f(its largest) for each of the lane's pieces that are all the row's; f(step, number of the first, keys) for
    // the steps in which that was true for some lane, and for the steps at the row's ends, whose pieces are never asked
    // for their largest. kAhead loads of a warp are on their way at once.
    template <class P, class F>
    __device__ void each_where(P piece_f, F f) const {
        constexpr int kAhead = 4;
        uint32_t key[Row<T>::kC];
        for (int32_t first = row.begin; first < row.end; first += kAhead) {
            if (first + kAhead <= row.end && row.inside(first) && row.inside(first + kAhead - 1)) {
                uint4 piece[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    piece[i] = __ldg(reinterpret_cast<const uint4*>(row.z + row.number(first + i, lane)));
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (!__any_sync(0xffffffffu, piece_f(largest_of<T>(piece[i])))) continue;
                    Row<T>::keys_of(piece[i], key);
                    f(first + i, row.number(first + i, lane), key);
                }
            } else {
                for (int32_t s = first; s < min(first + kAhead, row.end); ++s) {
                    const int32_t j = row.load(s, lane, key);
                    f(s, j, key);
                }
            }
        }
    }
    // f for every step.
    template <class F>
    __device__ void each(F f) const {
        each_where([](float) { return true; }, f);
    }

    __device__ void clear_histogram() {
        for (int b = tid; b < kBins; b += kThreads) sm.hist.count[b] = sm.hist.lo[b] = sm.hist.hi[b] = 0u;
        __syncthreads();
    }
    __device__ void put(int b, uint64_t w) {
        atomicAdd(&sm.hist.count[b], 1u);
        if (w == 0u) return;
        const uint32_t lo = static_cast<uint32_t>(w);
        const uint32_t old = atomicAdd(&sm.hist.lo[b], lo);
        const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
        if (hi) atomicAdd(&sm.hist.hi[b], hi);
    }
    // The cluster's histogram into `out` of every block: each block adds up a share of the bins, then all read them.
    __device__ void merge(Totals& out) {
        const int share = kBins / ranks;
        cluster.sync();
        for (int b = tid; b < share; b += kThreads) {
            uint64_t w = 0u;
            uint32_t n = 0u;
            for (int r = 0; r < ranks; ++r) {
                const Histogram* h = cluster.map_shared_rank(&sm.hist, r);
                const int at = rank * share + b;
                n += h->count[at];
                w += (static_cast<uint64_t>(h->hi[at]) << 32) + h->lo[at];
            }
            sm.merged.count[b] = n;
            sm.merged.weight[b] = w;
        }
        cluster.sync();
        for (int b = tid; b < kBins; b += kThreads) {
            const Totals* m = cluster.map_shared_rank(&sm.merged, b / share);
            out.count[b] = m->count[b % share];
            out.weight[b] = m->weight[b % share];
        }
        __syncthreads();
    }
    // The first bin at which the running count, or weight, reaches the target: found_bin, and what comes before it.
    // kBins - 1 where none does.
    __device__ void find_bin(const Totals& t, bool by_count, uint64_t target) {
        constexpr int kEach = kBins / kThreads;
        uint32_t n = 0u;
        uint64_t w = 0u;
        __syncthreads();  // the last answer has been read by all
#pragma unroll
        for (int i = 0; i < kEach; ++i) n += t.count[tid * kEach + i], w += t.weight[tid * kEach + i];
        uint64_t n_upto = warp_upto(n, lane), w_upto = warp_upto(w, lane);
        if (lane == 31) sm.sums[warp] = w_upto, sm.counts[warp] = static_cast<uint32_t>(n_upto);
        if (tid == 0) sm.found_bin = -1;
        __syncthreads();
        for (int i = 0; i < warp; ++i) n_upto += sm.counts[i], w_upto += sm.sums[i];
        uint64_t n_before = n_upto - n, w_before = w_upto - w;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int b = tid * kEach + i;
            const uint64_t n_to = n_before + t.count[b], w_to = w_before + t.weight[b];
            const bool reached = by_count ? n_to >= target : w_to >= target;
            const bool already = by_count ? n_before >= target : w_before >= target;
            if (b == kBins - 1 ? !already : reached && !already) {
                sm.found_bin = b;
                sm.before_count = static_cast<uint32_t>(n_before);
                sm.before_weight = w_before;
            }
            n_before = n_to;
            w_before = w_to;
        }
        __syncthreads();
    }
    // Sorts the block's list of n numbers: four to a thread in registers, compared there, with shuffles within 128 and
    // over shared memory beyond; 2048 take a quarter of the time that they take over shared memory alone, and up to 128
    // are one warp's.
    __device__ void sort_list(int n) {
        constexpr int kEach = kList / kThreads;
        static_assert(kEach == 4, "four to a thread");
        int size = 4;
        while (size < n) size <<= 1;
        __syncthreads();
        uint64_t v[kEach];
        const int first = tid * kEach;
        const bool mine = first < size;
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i] = first + i < n ? sm.list[first + i] : ~uint64_t{0};
        auto order = [](uint64_t& a, uint64_t& b, bool up) {
            const uint64_t lo = a < b ? a : b, hi = a < b ? b : a;
            a = up ? lo : hi;
            b = up ? hi : lo;
        };
        if (warp * 32 * kEach < size) order(v[0], v[1], true), order(v[2], v[3], false);
        for (int k = 4; k <= size; k <<= 1) {
            const bool up = (first & k) == 0;
            for (int j = k >> 1; j >= 32 * kEach; j >>= 1) {  // a thread's four meet another warp's four
                __syncthreads();
                if (mine) {
#pragma unroll
                    for (int i = 0; i < kEach; ++i) sm.list[first + i] = v[i];
                }
                __syncthreads();
                if (mine) {
                    const bool low = up == ((first & j) == 0);
#pragma unroll
                    for (int i = 0; i < kEach; ++i) {
                        const uint64_t other = sm.list[(first + i) ^ j];
                        v[i] = (v[i] < other) == low ? v[i] : other;
                    }
                }
            }
            if (warp * 32 * kEach >= size) continue;
            for (int j = min(k >> 1, 16 * kEach); j >= kEach; j >>= 1) {
                const bool low = up == ((first & j) == 0);
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const uint64_t other = __shfl_xor_sync(0xffffffffu, v[i], j / kEach);
                    v[i] = (v[i] < other) == low ? v[i] : other;
                }
            }
            order(v[0], v[2], up), order(v[1], v[3], up);
            order(v[0], v[1], up), order(v[2], v[3], up);
        }
        __syncthreads();
        if (mine) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) sm.list[first + i] = v[i];
        }
        __syncthreads();
    }
    // What comes before `own` in the order of the block's threads.
    __device__ uint64_t before_of(uint64_t own) {
        const uint64_t upto = warp_upto(own, lane);
        if (lane == 31) sm.sums[warp] = upto;
        __syncthreads();
        uint64_t before = upto - own;
        for (int i = 0; i < warp; ++i) before += sm.sums[i];
        __syncthreads();
        return before;
    }
    // The smallest key of the bins up to b, which is not the last one. Passes over the row compare keys with it, which
    // takes a third of the instructions that a token's bin does (256 x 131072 f32, top-p: 274 us against 295). Each warp
    // searches with 32 keys at a time, near the logit that the bin's number stands for (else seven steps of them took
    // 1 us).
    __device__ uint32_t least_key(int b) const {
        uint32_t below = 0u, key = order_key(weigh.max);  // a key of a later bin, and one of these
        const float at = weigh.max - static_cast<float>((b + 1) * (256 / kPerOctave)) / weigh.c_hi;
        const float off = (fabsf(weigh.max) + fabsf(at)) * 0x1p-20f, z_below = at - off, z_key = at + off;
        if (z_below < z_key && z_key < weigh.max && weigh.bin(z_below) > b && weigh.bin(z_key) <= b)
            below = order_key(z_below), key = order_key(z_key);
        while (key - below > 1u) {
            const uint32_t step = (key - below + 31u) / 32u;
            const uint32_t mine = min(static_cast<uint32_t>(lane + 1), (key - below) / step) * step + below;
            const uint32_t in = __ballot_sync(0xffffffffu, weigh.bin(key_value(mine)) <= b);
            const int first = in ? __ffs(in) - 1 : 31;
            const uint32_t from = __shfl_sync(0xffffffffu, mine, first > 0 ? first - 1 : 0), to = __shfl_sync(0xffffffffu, mine, first);
            if (first > 0) below = from;
            if (in) key = to;
            else below = to;
        }
        return key;
    }
    // The tokens for which which(key) holds go to the first block's list, as keys from the largest and numbers; listed
    // is their number, which may be more than the list holds. piece_may: of a piece's largest logit, whether it may have
    // one.
    template <class P, class F>
    __device__ void gather(P piece_may, F which) {
        if (tid == 0) sm.listed = 0u;
        __syncthreads();
        each_where(piece_may, [&](int32_t, int32_t j, const uint32_t (&key)[Row<T>::kC]) {
#pragma unroll
            for (int e = 0; e < Row<T>::kC; ++e)
                if (which(key[e])) {
                    const uint32_t at = atomicAdd(&sm.listed, 1u);
                    if (at < kList) sm.list[at] = (static_cast<uint64_t>(~key[e]) << 32) | static_cast<uint32_t>(j + e);
                }
        });
        cluster.sync();
        if (rank > 0) {  // to the end of the first block's list
            const uint32_t n = sm.listed;
            if (tid == 0) sm.before_count = atomicAdd(cluster.map_shared_rank(&sm.listed, 0), n);
            __syncthreads();
            uint64_t* list = cluster.map_shared_rank(sm.list, 0);
            const uint32_t at = sm.before_count;
            for (uint32_t i = tid; i < n && at + i < kList; i += kThreads) list[at + i] = sm.list[i];
        }
        cluster.sync();
    }
    // Sorts the first block's list of n tokens by key, then number, and cuts it where the target is reached.
    __device__ void cut_list(int n, bool by_count, uint64_t target, uint32_t before_count, uint64_t before_weight) {
        sort_list(n);
        constexpr int kEach = kList / kThreads;
        uint64_t w[kEach], own = 0u;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = tid * kEach + i;
            w[i] = at < n ? weigh(key_value(~static_cast<uint32_t>(sm.list[at] >> 32))) : 0u;
            own += w[i];
        }
        uint64_t before = before_weight + before_of(own);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = tid * kEach + i;
            const bool last = at == n - 1;
            const bool here = by_count ? before_count + at + 1 == target || (last && before_count + n < target)
                                       : before < target && (before + w[i] >= target || last);
            if (at < n && here) {
                sm.cut.key = ~static_cast<uint32_t>(sm.list[at] >> 32);
                sm.cut.last = static_cast<int32_t>(sm.list[at]);
                sm.cut_weight = before + w[i];
            }
            before += w[i];
        }
        __syncthreads();
    }
    // The first token, by number, at which the running sum of weight(key, number) over the row exceeds target(the
    // whole sum); `own` is this warp's part of the sum. Every block gets it (-1 where the sum never does), and the sum.
    template <class G, class F>
    __device__ int32_t search(uint64_t own, G target_of, F weight, uint64_t* whole) {
        if (lane == 0) sm.sums[warp] = own;
        __syncthreads();
        uint64_t before = 0u;
        if (tid == 0) {
            for (int i = 0; i < kWarps; ++i) before += sm.sums[i];
            sm.total = before;
            sm.chosen = -1;
        }
        cluster.sync();
        before = *whole = 0u;
        for (int r = 0; r < ranks; ++r) {
            const uint64_t part = *cluster.map_shared_rank(&sm.total, r);
            *whole += part;
            if (r < rank) before += part;
        }
        const uint64_t target = target_of(*whole);
        for (int i = 0; i < warp; ++i) before += sm.sums[i];
        if (before <= target && target < before + own) {  // one warp of the cluster
            // the run of steps, then the step
            const uint64_t run = sm.runs[warp][lane];
            const uint64_t run_upto = before + warp_upto(run, lane);
            const int at = __ffs(__ballot_sync(0xffffffffu, target < run_upto)) - 1;
            before = __shfl_sync(0xffffffffu, run_upto - run, at);
            for (int32_t s = row.begin + at * row.run; s < row.end; ++s) {
                uint32_t key[Row<T>::kC];
                const int32_t j = row.load(s, lane, key);
                uint64_t w[Row<T>::kC], mine = 0u;
#pragma unroll
                for (int e = 0; e < Row<T>::kC; ++e) mine += w[e] = weight(key[e], j + e);
                const uint64_t upto = warp_upto(mine, lane);
                const uint64_t step = __shfl_sync(0xffffffffu, upto, 31);
                if (target < before + step) {
                    before += upto - mine;
                    if (before <= target && target < before + mine) {
#pragma unroll
                        for (int e = 0; e < Row<T>::kC; ++e) {
                            if (before <= target && target < before + w[e]) sm.chosen = j + e;
                            before += w[e];
                        }
                    }
                    break;
                }
                before += step;
            }
        }
        cluster.sync();
        int32_t chosen = -1;
        for (int r = 0; r < ranks; ++r) chosen = max(chosen, *cluster.map_shared_rank(&sm.chosen, r));
        return chosen;
    }
    // The sum of the warps' parts over the cluster, to everyone.
    __device__ uint64_t cluster_total(uint64_t own) {
        if (lane == 0) sm.sums[warp] = own;
        __syncthreads();
        if (tid == 0) {
            own = 0u;
            for (int i = 0; i < kWarps; ++i) own += sm.sums[i];
            sm.total = own;
        }
        cluster.sync();
        uint64_t whole = 0u;
        for (int r = 0; r < ranks; ++r) whole += *cluster.map_shared_rank(&sm.total, r);
        cluster.sync();  // read by all before it is written again
        return whole;
    }
    // The sum of weight(key, number) over the warp's tokens, and over each of its runs of steps.
    template <class P, class F>
    __device__ uint64_t warp_sum_of(P piece_may, F weight) const {
        uint64_t mine = 0u, whole = 0u;
        int32_t run = 0, run_end = row.begin + row.run;
        sm.runs[warp][lane] = 0u;
        __syncwarp();
        auto close = [&] {
            mine = warp_total(mine);
            if (lane == 0) sm.runs[warp][run] = mine;
            whole += mine;
            mine = 0u;
        };
        each_where(piece_may, [&](int32_t s, int32_t j, const uint32_t (&key)[Row<T>::kC]) {
            if (s >= run_end) {
                close();
                while (s >= run_end) run_end += row.run, ++run;
            }
#pragma unroll
            for (int e = 0; e < Row<T>::kC; ++e) mine += weight(key[e], j + e);
        });
        close();
        __syncwarp();
        return whole;
    }
    // All of the choice by the first block, from its list of the n tokens that come first in the order.
    struct Filters {
        uint64_t top_k;   // n or less
        uint64_t share;   // top_p in units of 2^-64, of `all` or of the first top_k's weight; 0 with !by_p
        uint64_t all;
        uint32_t least;   // the smallest key that min_p keeps
        bool by_k, by_p;
    };
    __device__ void choose_from_list(int n, const Filters& f, float u, uint64_t* total, int32_t* token) {
        constexpr int kEach = kList / kThreads;
        sort_list(n);
        if (tid == 0) sm.listed = static_cast<uint32_t>(min(static_cast<uint64_t>(n), f.top_k));
        uint64_t w[kEach], own = 0u;
        uint32_t key[kEach];
        int32_t number[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = tid * kEach + i;
            key[i] = at < n ? ~static_cast<uint32_t>(sm.list[at] >> 32) : 0u;
            number[i] = at < n ? static_cast<int32_t>(sm.list[at]) : 0;
            w[i] = at < n ? weigh(key_value(key[i])) : 0u;
            own += w[i];
        }
        const uint64_t before = before_of(own);
        // the weight of the first `listed` of them, to everyone
        auto weight_upto_listed = [&] {
            const int m = static_cast<int>(sm.listed);
            uint64_t run = before;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                run += w[i];
                if (tid * kEach + i == m - 1) sm.cut_weight = run;
            }
            __syncthreads();
            return sm.cut_weight;
        };
        if (f.by_p) {
            const uint64_t base = f.by_k ? weight_upto_listed() : f.all;
            const uint64_t need = share_of(f.share, base);
            uint64_t run = before;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (run < need && run + w[i] >= need) atomicMin(&sm.listed, static_cast<uint32_t>(tid * kEach + i + 1));
                run += w[i];
            }
            __syncthreads();
        }
        if (f.least > 1u) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (tid * kEach + i > 0 && key[i] < f.least) atomicMin(&sm.listed, static_cast<uint32_t>(tid * kEach + i));
            __syncthreads();
        }
        *total = weight_upto_listed();
        const int m = static_cast<int>(sm.listed);
        // the kept ones by number
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (tid * kEach + i < m) sm.list[tid * kEach + i] = (static_cast<uint64_t>(number[i]) << 32) | key[i];
        __syncthreads();
        sort_list(m);
        own = 0u;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = tid * kEach + i;
            w[i] = at < m ? weigh(key_value(static_cast<uint32_t>(sm.list[at]))) : 0u;
            own += w[i];
        }
        const uint64_t place = place_of(u, *total);
        uint64_t run = before_of(own);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (run <= place && place < run + w[i]) sm.chosen = static_cast<int32_t>(sm.list[tid * kEach + i] >> 32);
            run += w[i];
        }
        __syncthreads();
        *token = sm.chosen;
    }
    // A number in [0, 1) as a place in a sum.
    __device__ static uint64_t place_of(float u, uint64_t total) {
        // u is m 2^(e - 150) with a 24-bit m; as a 64-bit fraction, cut off below 2^-64
        u = u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
        const int e = static_cast<int>(__float_as_uint(u) >> 23);
        const uint64_t m = (__float_as_uint(u) & 0x7fffffu) | (e > 0 ? 0x800000u : 0u);
        const int up = (e > 0 ? e : 1) - 150 + 64;
        return __umul64hi(up >= 0 ? m << up : up > -24 ? m >> -up : 0u, total);
    }
    // The cut at which the running count (or weight) of the order reaches the target, and the weight up to it.
    __device__ Cut select(bool by_count, uint64_t target, uint64_t* upto) {
        find_bin(sm.first, by_count, target);
        const int bin = sm.found_bin;
        uint32_t before_count = sm.before_count;
        uint64_t before_weight = sm.before_weight;
        // the last bin was not counted: it holds what is left of the row
        uint32_t n = bin == kBins - 1 ? static_cast<uint32_t>(row.V) - before_count : sm.first.count[bin];
        // the keys that are still in question
        uint32_t lo = bin == kBins - 1 ? 1u : least_key(bin), hi = bin == 0 ? order_key(weigh.max) : least_key(bin - 1) - 1u;
        auto within = [&](uint32_t key) { return key >= lo && key <= hi; };
        while (n > kList && lo < hi) {
            const int by = max(0, 22 - __clz(hi - lo));
            clear_histogram();
            each([&](int32_t, int32_t, const uint32_t (&key)[Row<T>::kC]) {
#pragma unroll
                for (int e = 0; e < Row<T>::kC; ++e)
                    if (within(key[e])) put(kBins - 1 - static_cast<int>((key[e] - lo) >> by), weigh(key_value(key[e])));
            });
            merge(sm.split);
            find_bin(sm.split, by_count, by_count ? target - before_count : target - before_weight);
            const uint32_t part = static_cast<uint32_t>(kBins - 1 - sm.found_bin);
            n = sm.split.count[sm.found_bin];
            before_count += sm.before_count;
            before_weight += sm.before_weight;
            const uint64_t top = lo + ((static_cast<uint64_t>(part) + 1u) << by) - 1u;
            lo += part << by;
            hi = top < hi ? static_cast<uint32_t>(top) : hi;
        }
        if (n > kList) {  // equal logits: the first of them by number
            const uint64_t each_weight = weigh(key_value(lo));
            uint64_t take = n;
            if (by_count) take = min(take, target - before_count);
            else if (each_weight > 0u) take = min(take, (target - before_weight + each_weight - 1u) / each_weight);
            auto one = [&](uint32_t key, int32_t) { return key == lo ? uint64_t{1} : uint64_t{0}; };
            *upto = before_weight + take * each_weight;
            uint64_t ties;
            const int32_t last =
                search(warp_sum_of([](float) { return true; }, one), [&](uint64_t) { return take - 1u; }, one, &ties);
            cluster.sync();  // read by all before it is written again
            return Cut{lo, last};
        }
        gather([&](float z) { return order_key(z) >= lo; }, within);
        if (rank == 0) cut_list(static_cast<int>(n), by_count, target, before_count, before_weight);
        cluster.sync();
        *upto = *cluster.map_shared_rank(&sm.cut_weight, 0);
        const Cut cut = *cluster.map_shared_rank(&sm.cut, 0);
        cluster.sync();  // read by all before it is written again
        return cut;
    }
};

// kWide: V is kWideV or more.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) k_sample(const T* __restrict__ logits, const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    SampleSmem& sm = *reinterpret_cast<SampleSmem*>(raw);
    Sampler<T> s{sm, cg::this_cluster()};
    s.rank = static_cast<int>(s.cluster.block_rank());
    s.ranks = static_cast<int>(s.cluster.num_blocks());
    s.tid = threadIdx.x;
    s.lane = s.tid & 31;
    s.warp = s.tid >> 5;
    const int64_t t = blockIdx.x / s.ranks;
    if (s.tid < 256) sm.table[s.tid] = kExp2Table[s.tid];
    Row<T>& row = s.row;
    row.z = logits + t * a.V;
    row.V = a.V;
    row.lead = static_cast<int>(reinterpret_cast<uintptr_t>(row.z) / sizeof(T) % Row<T>::kC);
    {  // steps in equal runs over the blocks, and over a block's warps
        const int32_t steps = static_cast<int32_t>((static_cast<int64_t>(a.V) + row.lead + Row<T>::kStep - 1) / Row<T>::kStep);
        const int32_t per_block = (steps + s.ranks - 1) / s.ranks, per_warp = (per_block + kWarps - 1) / kWarps;
        const int32_t block_end = min(steps, (s.rank + 1) * per_block);
        row.begin = min(block_end, s.rank * per_block + s.warp * per_warp);
        row.end = min(block_end, row.begin + per_warp);
        row.run = (per_warp + 31) / 32;
    }
    griddep_wait();
    griddep_launch_dependents();
    const float tau = a.temperature ? a.temperature[t] : 1.0f, least = a.min_p ? a.min_p[t] : 0.0f;
    // the largest logit
    uint32_t top = 0u;
    s.each_where(
        [&](float z) {
            top = max(top, order_key(z));
            return false;
        },
        [&](int32_t, int32_t, const uint32_t (&key)[Row<T>::kC]) {
#pragma unroll
            for (int e = 0; e < Row<T>::kC; ++e) top = max(top, key[e]);
        });
    // of the cluster's, the largest of every block's v
    auto cluster_max = [&](uint32_t v) {
        v = __reduce_max_sync(0xffffffffu, v);
        if (s.lane == 0) sm.counts[s.warp] = v;
        __syncthreads();
        if (s.tid == 0) {
            for (int i = 1; i < kWarps; ++i) v = max(v, sm.counts[i]);
            sm.best = v;
        }
        s.cluster.sync();
        for (int r = 0; r < s.ranks; ++r) v = max(v, *s.cluster.map_shared_rank(&sm.best, r));
        return v;
    };
    top = cluster_max(top);
    const float largest = key_value(top);
    const bool speaks = s.rank == 0 && s.tid == 0;
    // nothing to choose: a logit that is not a number, or nothing but -inf
    const bool none = top == 0xffffffffu || largest == -INFINITY;
    if (none || !(tau > 0x1p-60f) || least > 1.0f) {  // no weight reaches a min_p above 1: the first of the order alone
        uint32_t first = 0u;  // the largest's first token, counted down from 2^32 - 1
        if (!none) {
            s.each_where([&](float z) { return order_key(z) == top; },
                         [&](int32_t, int32_t j, const uint32_t (&key)[Row<T>::kC]) {
#pragma unroll
                             for (int e = 0; e < Row<T>::kC; ++e)
                                 if (key[e] == top) first = max(first, 0xffffffffu - static_cast<uint32_t>(j + e));
                         });
            s.cluster.sync();  // the last maximum has been read
            first = cluster_max(first);
        }
        if (speaks) {
            a.token[t] = none ? -1 : static_cast<int32_t>(0xffffffffu - first);
            if (a.logprob) a.logprob[t] = none ? NAN : 0.0f;
        }
        s.cluster.sync();  // nobody leaves while another may read its memory
        return;
    }
    const int32_t k = a.top_k ? a.top_k[t] : 0;
    const float p = a.top_p ? a.top_p[t] : 1.0f;
    const bool by_k = k > 0 && k < a.V, by_p = p < 1.0f;
    if (s.tid == 0) {  // the 64-bit arithmetic, of which an SM has little
        const double c = 256.0 * 1.4426950408889634 / static_cast<double>(tau);
        sm.c_hi = static_cast<float>(c);
        sm.c_lo = static_cast<float>(c - static_cast<double>(sm.c_hi));
        sm.share = by_p && p > 0.0f ? static_cast<uint64_t>(static_cast<double>(p) * 0x1p64) : 0u;
        // min_p keeps the logits whose weight is min_p of the largest; the largest always stays
        sm.least = 1u;
        if (least > 0.0f && !isinf(tau)) {
            const double at = static_cast<double>(largest) + static_cast<double>(tau) * log(static_cast<double>(least));
            sm.least = order_key(at < static_cast<double>(largest) ? __double2float_ru(at) : largest);
        }
    }
    __syncthreads();
    s.weigh = Weigh{sm.table, largest, sm.c_hi, sm.c_lo, a.shift};
    const Weigh& weigh = s.weigh;
    if constexpr (kWide) {
        // A row whose weights are mostly small gets units as fine as a sum below 2^62 allows. In units of 2^-a.shift each
        // weight loses less than one, so that all + V bounds the sum in finer ones.
        const uint64_t all = s.cluster_total(
            s.warp_sum_of([](float) { return true; }, [&](uint32_t key, int32_t) { return weigh(key_value(key)); }));
        s.weigh.shift = min(61, a.shift + __clzll(static_cast<long long>(all + static_cast<uint64_t>(a.V))) - 2);
    }
    const uint32_t least_key = sm.least;
    const uint64_t share = sm.share;
    const float u = a.uniform[t];
    Cut cut{least_key, 0x7fffffff};
    uint64_t total = 0u;
    int32_t token = -1;
    bool done = false;
    if (by_k || by_p) {
        // Counts are enough to find the first top_k, shares need the weights too.
        auto count = [&](bool weights) {
            s.clear_histogram();
            s.each([&](int32_t, int32_t, const uint32_t (&key)[Row<T>::kC]) {
#pragma unroll
                for (int e = 0; e < Row<T>::kC; ++e) {
                    const float z = key_value(key[e]);
                    const int b = key[e] == 0u ? kBins - 1 : weigh.bin(z);
                    // the last bin's weights are 0, its count is what is left
                    if (b < kBins - 1) s.put(b, weights ? weigh(z) : 0u);
                }
            });
            s.merge(sm.first);
        };
        auto all_weights = [&] {
            uint64_t w = 0u;
            for (int b = s.tid; b < kBins; b += kThreads) w += sm.first.weight[b];
            w = warp_total(w);
            __syncthreads();
            if (s.lane == 0) sm.sums[s.warp] = w;
            __syncthreads();
            w = 0u;
            for (int i = 0; i < kWarps; ++i) w += sm.sums[i];
            __syncthreads();
            return w;
        };
        // The first top_k tokens have logits of at least the top_k'th largest of the pieces' largest ones: enough to
        // list them, with few others, at an eighth (a quarter) of the counting.
        int bin = kBins - 1;
        uint32_t upto = 0u;
        uint64_t kept = 0u;
        bool listed = false;
        if (by_k) {
            s.clear_histogram();
            s.each_where(
                [&](float z) {
                    const int b = weigh.bin(z);
                    if (b < kBins - 1) s.put(b, 0u);
                    return false;
                },
                [&](int32_t, int32_t, const uint32_t (&key)[Row<T>::kC]) {
#pragma unroll
                    for (int e = 0; e < Row<T>::kC; ++e) {
                        const int b = key[e] == 0u ? kBins - 1 : weigh.bin(key_value(key[e]));
                        if (b < kBins - 1) s.put(b, 0u);
                    }
                });
            s.merge(sm.first);
            s.find_bin(sm.first, true, static_cast<uint64_t>(k));
            bin = sm.found_bin;
        } else {
            count(true);
            kept = all_weights();
            s.find_bin(sm.first, false, share_of(share, kept));
            bin = sm.found_bin;
            if (sm.before_count + sm.first.count[bin] > kList) bin = kBins - 1;
        }
        if (bin < kBins - 1) {
            const uint32_t from = s.least_key(bin);
            s.gather([&](float z) { return order_key(z) >= from; }, [&](uint32_t key) { return key >= from; });
            upto = *s.cluster.map_shared_rank(&sm.listed, 0);
            listed = upto <= kList;
            s.cluster.sync();  // read before the first block counts in it again
        }
        if (listed) {  // the first block does the rest
            if (s.rank == 0)
                s.choose_from_list(static_cast<int>(upto),
                                   {by_k ? static_cast<uint64_t>(k) : ~uint64_t{0}, share, kept, least_key, by_k, by_p}, u,
                                   &total, &token);
            done = true;
        } else {
            if (by_k) {
                count(by_p);
                const Cut at = s.select(true, static_cast<uint64_t>(k), &kept);
                if (at.key >= cut.key) cut = at;
            }
            if (by_p) {
                const Cut at = s.select(false, share_of(share, kept), &kept);
                if (at.key > cut.key || (at.key == cut.key && at.last < cut.last)) cut = at;
            }
        }
    }
    if (!done) {
        auto kept_weight = [&](uint32_t key, int32_t j) -> uint64_t {
            return key > cut.key || (key == cut.key && j <= cut.last) ? weigh(key_value(key)) : 0u;
        };
        const uint64_t own = s.warp_sum_of([&](float z) { return order_key(z) >= cut.key; }, kept_weight);
        token = s.search(own, [&](uint64_t all) { return Sampler<T>::place_of(u, all); }, kept_weight, &total);
    }
    if (speaks) {
        a.token[t] = token;
        if (a.logprob) {
            const float z = to_float(row.z[token]);
            const double x = z == largest ? 0.0 : (static_cast<double>(z) - static_cast<double>(largest)) / static_cast<double>(tau);
            a.logprob[t] = static_cast<float>(x - log(ldexp(static_cast<double>(total), -weigh.shift)));
        }
    }
    s.cluster.sync();  // nobody leaves while another may read its memory
}

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

template <typename T, bool kWide>
cudaError_t run(const SampleProblem& p, const SampleArgs& a, cudaStream_t stream) {
    cudaError_t e = allow_smem<&k_sample<T, kWide>>(sizeof(SampleSmem));
    if (e != cudaSuccess) return e;
    // blocks to a row: two to an SM in all, each with at least 2048 tokens
    int ranks = 8;
    while (ranks > 1 && (p.T * ranks > 2 * static_cast<int64_t>(p.sm_count) || p.V / ranks < 2048)) ranks /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.T * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(SampleSmem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_sample<T, kWide>, static_cast<const T*>(p.logits), a);
}

}  // namespace

moe_status_t launch_sample(const SampleProblem& p, cudaStream_t stream) {
    SampleArgs a{p.uniform, p.temperature, p.top_p, p.min_p, p.top_k, p.token, p.logprob, p.V, kShift};
    if (p.V >= kWideV)
        while ((p.V >> (62 - a.shift)) > 0) --a.shift;  // V of the largest weight stay below 2^62
    auto of_type = [&](auto t) {
        using T = decltype(t);
        return p.V >= kWideV ? run<T, true>(p, a, stream) : run<T, false>(p, a, stream);
    };
    const cudaError_t e = p.dtype == MOE_DTYPE_F32    ? of_type(float{})
                          : p.dtype == MOE_DTYPE_BF16 ? of_type(__nv_bfloat16{})
                                                      : of_type(__half{});
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
