// Draw of the next token from logits: temperature, top-k, top-p, min-p.
//
//   w_i = exp((l_i - max l) / T) held as the whole number floor(2^40 w_i);
//   kept: rank < top_k, mass before < top_p * mass of the top_k, w_i >= min_p;
//   token: the first index whose sum of kept mass exceeds floor(u * kept mass).
//
// Whole-number masses add up to the same sum in any order (a row holds less
// than 2^59), so histograms with atomics, any split of the row and any order of
// arrival give the same token. What lies above a threshold is told by logit and
// index in some variants, by the bits of the weights first in others: the same
// set, for expf never falls as its argument rises (looked at for every float32
// from -110 to 0) and the steps before it are rounded to nearest.
//
// A row is one cluster's: its CTAs exchange maxima, histograms and sums through distributed shared memory. top-k and top-p
// are thresholds in the order (logit falling, index rising), and what lies above one is nearly always few tokens:
//   - top_k: the largest logit of every thread is counted in a histogram. The bin where the count reaches k bounds the k
//     largest of all from below, and little more than k logits lie above it.
//   - top_p alone: a histogram of the masses by the leading bits of the weights, and one by the next bits inside the bin that
//     the threshold lies in.
// The first CTA ranks these candidates and draws among them, or tells the others the threshold. Rows where too many
// candidates are left (flat ones, many equal logits) are resolved bin by bin, then bit by bit, then by index.
//
// The bound of few rows is latency: the exchanges, and instructions that run once and have to be fetched. 16 CTAs a row
// (8 from 9 rows on) read it once and keep it in shared memory: 1 x 151,936 with top_k 20 8.6 us, 16 x 151,936 bfloat16
// with top_p 0.9 38 us. The bound of many rows is the time that a row's steps hold an SM, so that the fewest CTAs that fill
// the GPU take a row and read it again from the L2 cache where they need it, for parts of rows in shared memory leave no
// room for other rows: 256 x 100,277 with top_k 50 in 31 us, 3.3 TB/s, where 8 CTAs each that keep the row took 85 us. What
// top_p alone costs there (256 x 151,936 bfloat16 282 us, 107 without any limit) is an exponential and two additions in
// shared memory a logit.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>
#include <utility>

#include "../../include/qmm.h"
#include "qmm_device.cuh"

namespace qmmk {

namespace {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kBins = 256;                 // few: every CTA reads every other's histogram, at shared memory's remote rate
constexpr int kList = 2048;                // candidates of the first CTA
constexpr int kEach = kList / kSampleThreads;
constexpr int kRanks = 16;                 // CTAs of a cluster at most
constexpr int kPortableRanks = 8;
constexpr int kManyCtas = 2 * 152;         // CTAs that the GPU holds at once
constexpr int kCounted = 256;              // candidates that are ranked by counting all others (kBins at most)
constexpr int kFew = 64;                   // the same where more have been parted by histograms
constexpr float kBinsPerUnit = 8.0f;       // bins for one unit of (max l - l) / T: mass ends at 27.7 units
constexpr int kWeightBinShift = 20;        // bits of a weight below its bin: 8 bins an octave

typedef unsigned long long u64;

struct SampleParams {
    const void* logits;
    int64_t stride;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* tokens;
    float* probs;
    int32_t vocab;
};

// What one level of a selection decided.
struct Decision {
    u64 mass;        // mass ranked before the bin
    u64 total;       // mass of everything that takes part
    u64 limit;       // what the mass before a kept element is below
    uint32_t count;  // elements ranked before the bin
    uint32_t bin;
    uint32_t members;
};

struct Threshold {   // kept: key > key, or key == key and index <= index
    uint32_t key;
    uint32_t index;
};

struct SampleShared {
    u64 sum[kRanks];
    float top[kRanks], level[kRanks], above[kRanks];
    u64 warp_mass[kSampleWarps];
    alignas(16) u64 mass[kBins];
    alignas(16) uint32_t count[kBins];
    uint32_t warp_count[kSampleWarps];
    u64 list[kList];
    u64 few[kFew], few_value[kFew], pick, pick_value;
    uint32_t own[kList];   // slots of this CTA's candidates
    u64 scalar;
    uint32_t list_size, sizes[kRanks], hit_count;
    uint16_t hits[kSampleThreads];
    Decision decision;
    Threshold threshold;
};

// Unsigned numbers in the order of the floats; NaN is -infinity, and -0 is 0.
__device__ __forceinline__ float clean(float l) { return fmaxf(l, -INFINITY) + 0.0f; }
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// (logit, index) as one number that falls along the ranks.
__device__ __forceinline__ u64 entry_of(uint32_t key, uint32_t index) {
    return static_cast<u64>(key) << 32 | (0xFFFFFFFFu - index);
}

template <class T>
__device__ __forceinline__ T warp_add(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
template <class T>
__device__ __forceinline__ T warp_scan(T v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T a = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += a;
    }
    return v;
}

// Sum of v over the threads before this one; `all`: over all. scratch: kSampleWarps numbers.
template <class N>
__device__ __forceinline__ N block_before(N v, N* scratch, N& all) {
    static_assert(kSampleWarps == 16, "half a warp scans the warps");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const N upto = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) scratch[warp] = upto;
    __syncthreads();
    const N mine = scratch[lane & 15];
    N w = mine;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        const N a = __shfl_up_sync(0xFFFFFFFFu, w, o, 16);
        if ((lane & 15) >= o) w += a;
    }
    all = __shfl_sync(0xFFFFFFFFu, w, 15);
    return upto - v + __shfl_sync(0xFFFFFFFFu, w - mine, warp);
}

// 64-bit sums of two 32-bit atomics each: a 64-bit one in shared memory is a loop of compare-and-swaps (37 a thread of
// 512 took 12,000 cycles, these 3,500).
__device__ __forceinline__ void add_mass(u64* sum, u64 m) {
    uint32_t* const w = reinterpret_cast<uint32_t*>(sum);
    const uint32_t lo = static_cast<uint32_t>(m), old = atomicAdd(&w[0], lo);
    const uint32_t hi = static_cast<uint32_t>(m >> 32) + (old + lo < old ? 1u : 0u);
    if (hi != 0) atomicAdd(&w[1], hi);
}

// The least whole number whose double is not below `limit`: `(double)a < limit` for whole a is `a < bound`. One thread's
// work (double arithmetic is slow on this GPU).
__device__ __forceinline__ u64 bound_of(double limit) {
    u64 a = static_cast<u64>(limit);
    if (a < (1ull << 53)) return static_cast<double>(a) < limit ? a + 1 : a;
    u64 lo = a - 4096, hi = a + 4096;   // conversions of numbers below 2^60 are off by 64 at most
    while (lo < hi) {
        const u64 mid = lo + (hi - lo) / 2;
        if (static_cast<double>(mid) < limit) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// HELD: the CTA keeps its part of the row in shared memory; else it reads it again in every pass.
template <class T, bool HELD>
struct RowSampler {
    // slots of a chunk: 16 bytes of the row in memory, or of the slots in shared memory
    static constexpr int kVec = HELD ? 4 : 16 / sizeof(T);
    static constexpr int kPerRead = 16 / static_cast<int>(sizeof(T)) / kVec;   // chunks of 16 bytes in memory
    SampleShared& sh;
    float* x;              // HELD: this CTA's slots, the logits and later their weights
    const T* src;          // the row
    int lo, hi;            // the slots that hold logits; those before and after in the first and the last chunk are -infinity
    int chunks;            // of the slots
    int shift;             // index of slot 0
    int rank, ranks;
    float top, temperature;
    Threshold thr;

    __device__ __forceinline__ float logit_at(uint32_t index) const {   // from memory
        if constexpr (sizeof(T) == 2)
            return clean(__uint_as_float(static_cast<uint32_t>(src[index]) << 16));
        else
            return clean(src[index]);
    }
    __device__ __forceinline__ uint32_t index(int i) const { return static_cast<uint32_t>(shift + i); }
    __device__ __forceinline__ float slot(int i) const {
        if constexpr (HELD) return x[i];
        else return i >= lo && i < hi ? logit_at(index(i)) : -INFINITY;   // an index outside the row is not one of memory
    }
    __device__ __forceinline__ static float pick(const float (&v)[kVec], int e) {
        float x = v[0];
#pragma unroll
        for (int k = 1; k < kVec; ++k) x = e == k ? v[k] : x;
        return x;
    }
    __device__ __forceinline__ bool inside(int c) const { return c * kVec >= lo && (c + 1) * kVec <= hi; }
    __device__ __forceinline__ uint4 raw(int c) const { return __ldg(reinterpret_cast<const uint4*>(src + shift + c * kVec)); }
    __device__ __forceinline__ static void unpack(const uint4& r, float (&v)[kVec]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            if constexpr (sizeof(T) == 2)
                v[e] = clean(__uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16));
            else
                v[e] = clean(__uint_as_float(w[e]));
        }
    }
    // The slots of chunk c.
    __device__ __forceinline__ void load(int c, float (&v)[kVec]) const {
        if constexpr (HELD) {
            const float4 f = *reinterpret_cast<const float4*>(x + c * kVec);
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else if (inside(c)) {
            unpack(raw(c), v);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const int i = c * kVec + e;
                v[e] = i >= lo && i < hi ? logit_at(index(i)) : -INFINITY;
            }
        }
    }
    // f(c, v) for chunks c = from, from + step, ... below end and their slots v.
    template <class F>
    __device__ __forceinline__ void each_chunk(int from, int end, int step, F f) const {
        if constexpr (HELD) {
            for (int c = from; c < end; c += step) {
                float v[kVec];
                load(c, v);
                f(c, v);
            }
        } else {
            for (int c0 = from; c0 < end; c0 += 4 * step) {   // four loads in flight
                uint4 r[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j * step < end && inside(c0 + j * step)) r[j] = raw(c0 + j * step);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = c0 + j * step;
                    if (c >= end) continue;
                    float v[kVec];
                    if (inside(c)) unpack(r[j], v);
                    else load(c, v);
                    f(c, v);
                }
            }
        }
    }
    // The chunks that the threads with `here` have read first (theirs are the 16 bytes at tid, tid + kSampleThreads, ...). All
    // threads call it, with sh.hit_count zero; where many chunks come from memory, a warp takes one such thread's at a time.
    template <class F>
    __device__ __forceinline__ void each_chunk_of(bool here, F f) const {
        const int reads = chunks / kPerRead;
        if (HELD || reads <= 8 * kSampleThreads) {
            if (!here) return;
            for (int r = threadIdx.x; r < reads; r += kSampleThreads) {
#pragma unroll
                for (int k = 0; k < kPerRead; ++k) {
                    float v[kVec];
                    load(r * kPerRead + k, v);
                    f(r * kPerRead + k, v);
                }
            }
            return;
        }
        if (here) sh.hits[atomicAdd(&sh.hit_count, 1u)] = static_cast<uint16_t>(threadIdx.x);
        __syncthreads();
        const int hits = static_cast<int>(sh.hit_count), lane = threadIdx.x & 31;
        for (int h = threadIdx.x >> 5; h < hits; h += kSampleWarps)
            each_chunk(sh.hits[h] + lane * kSampleThreads, reads, 32 * kSampleThreads, f);
    }
    __device__ __forceinline__ float depth(float l) const { return temperature == 1.0f || l == top ? l == top ? 0.0f : l - top : __fdiv_rn(l - top, temperature); }
    __device__ __forceinline__ float weight(float l, float z) const { return l == top ? 1.0f : expf(z); }
    __device__ __forceinline__ float weight(float l) const { return weight(l, depth(l)); }
    // floor(2^40 w) from the bits of w, for conversions to 64 bits run at the rate of double arithmetic. 0 also where an
    // infinite temperature or logit leaves no number.
    __device__ __forceinline__ static u64 mass(float w) {
        const uint32_t b = __float_as_uint(w), at = 133u - (b >> 23);   // 6 for 1, 46 for 2^-40
        const u64 m = (static_cast<u64>((b & 0x7FFFFFu) | 0x800000u) << 23) >> (at & 63u);
        return at - 6u <= 40u ? m : 0ull;
    }
    // The weights of a chunk, without branches between its slots.
    __device__ __forceinline__ void weights(const float (&v)[kVec], float (&w)[kVec]) const {
#pragma unroll
        for (int e = 0; e < kVec; ++e) w[e] = v[e] == top ? 0.0f : v[e] - top;
        if (temperature != 1.0f) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[e] = __fdiv_rn(w[e], temperature);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) w[e] = expf(w[e]);
    }
    __device__ __forceinline__ bool under(uint32_t key, uint32_t idx) const {
        return key > thr.key || (key == thr.key && idx <= thr.index);
    }

    // ---- candidates ------------------------------------------------------------------------------------------------

    // Every CTA has a part of the first one's list for its own candidates.
    __device__ __forceinline__ void clear_list() {
        if (threadIdx.x == 0) sh.list_size = sh.hit_count = 0u;
    }
    __device__ __forceinline__ void add(uint32_t key, uint32_t index) {
        const uint32_t room = kList / ranks, at = atomicAdd(&sh.list_size, 1u);
        if (at < room) cg::this_cluster().map_shared_rank(&sh, 0)->list[rank * room + at] = entry_of(key, index);
    }

    // The number of candidates of all CTAs, which the first one then has in its list; more than kList where a CTA had more
    // than fit its part. All CTAs call it, and are done with one another's memory after it.
    __device__ int collect() {
        cg::cluster_group cluster = cg::this_cluster();
        __syncthreads();
        if (threadIdx.x < ranks) cluster.map_shared_rank(&sh, threadIdx.x)->sizes[rank] = sh.list_size;
        cluster.sync();
        const uint32_t room = kList / ranks, lane = threadIdx.x & 31;
        const uint32_t size = lane < ranks ? sh.sizes[lane] : 0u, n = __reduce_add_sync(0xFFFFFFFFu, size);
        const bool fits = __all_sync(0xFFFFFFFFu, size <= room);
        if (!fits) return kList + 1;
        if (rank == 0 && ranks > 1) {   // close the gaps
            u64 e[kList / kSampleThreads];
#pragma unroll
            for (int k = 0; k < kList / kSampleThreads; ++k) {
                const uint32_t i = threadIdx.x + k * kSampleThreads;
                if (i >= n) break;
                uint32_t at = i;
                int r = 0;
                while (at >= sh.sizes[r]) at -= sh.sizes[r++];
                e[k] = sh.list[r * room + at];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kList / kSampleThreads; ++k) {
                const uint32_t i = threadIdx.x + k * kSampleThreads;
                if (i < n) sh.list[i] = e[k];
            }
        }
        __syncthreads();
        return static_cast<int>(n);
    }

    // One thread's result for all; a barrier before and after.
    template <class F>
    __device__ __forceinline__ u64 by_one(F f) {
        __syncthreads();
        if (threadIdx.x == 0) sh.scalar = f();
        __syncthreads();
        return sh.scalar;
    }
    __device__ __forceinline__ static u64 mass_limit(float top_p, u64 total) {
        return bound_of(static_cast<double>(top_p) * static_cast<double>(total));
    }
    __device__ __forceinline__ static u64 target_of(float u, u64 total) {
        const double want = static_cast<double>(u) * static_cast<double>(total);
        const u64 target = want > 0.0 ? static_cast<u64>(want) : 0ull;
        return target >= total ? total - 1 : target;
    }

    // The draw among the n candidates of the list, which hold everything that may be kept; by the first CTA. `total`: the
    // mass that top_p is a share of, 0 where it is that of the top_k candidates.
    __device__ void finish(const SampleParams& p, int row, int n, int top_k, float top_p, float min_p, u64 total) {
        const int k = top_k > 0 && top_k < n ? top_k : n;
        if (n <= kCounted) finish_counted(p, row, n, k, top_p, min_p, total);
        else finish_parted(p, row, n, k, top_p, min_p, total);
    }

    // Every candidate counts those that rank before it, and then those of lower indices.
    __device__ __forceinline__ void finish_counted(const SampleParams& p, int row, int n, int k, float top_p, float min_p,
                                                   u64 total) {
        const int tid = threadIdx.x;
        const u64 e = tid < n ? sh.list[tid] : 0ull;
        const float w = tid < n ? weight(value_of(static_cast<uint32_t>(e >> 32))) : 0.0f;
        u64 m = mass(w), all;
        if (tid < kCounted) sh.mass[tid] = m;   // the histogram is used up
        __syncthreads();
        int place = 0;
        u64 before = 0;
        if (tid < n) {
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                const bool first = sh.list[j] > e;
                place += first ? 1 : 0;
                before += first ? sh.mass[j] : 0ull;
            }
        }
        bool keep = tid < n && place < k && !(w < min_p);
        if (top_p < 1.0f) {
            if (total == 0) (void)block_before(place < k ? m : 0ull, sh.warp_mass, total);
            keep &= before < by_one([&] { return mass_limit(top_p, total); });
        }
        m = keep ? m : 0ull;
        __syncthreads();
        if (tid < kCounted) sh.mass[tid] = m;
        (void)block_before(m, sh.warp_mass, all);
        const u64 target = by_one([&] { return target_of(p.u[row], all); });
        if (m == 0) return;
        const uint32_t low = static_cast<uint32_t>(e);   // falls with the index
        before = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) before += static_cast<uint32_t>(sh.list[j]) > low ? sh.mass[j] : 0ull;
        if (target >= before && target < before + m) {
            p.tokens[row] = static_cast<int32_t>(0xFFFFFFFFu - low);
            if (p.probs != nullptr) p.probs[row] = __fdiv_rn(static_cast<float>(m), static_cast<float>(all));
        }
    }

    // Of the elements whose bits of `in` are set, the last one in the order of falling `order` (all different) whose values
    // before it add up to less than `limit`, which is not 0; to sh.pick. Histograms of 256 parts of the elements' range,
    // then of the part that it lies in, until that has few. (Sorting 2,048 entries took 11 us, this takes 1 to 2.)
    __device__ __forceinline__ void last_below(const u64 (&order)[kEach], const u64 (&value)[kEach], uint32_t in, u64 limit) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        uint32_t top = 0u, low = 0xFFFFFFFFu;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (!(in >> k & 1)) continue;
            top = max(top, static_cast<uint32_t>(order[k] >> 32));
            low = min(low, static_cast<uint32_t>(order[k] >> 32));
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        low = __reduce_min_sync(0xFFFFFFFFu, low);
        __syncthreads();
        if (lane == 0) {
            sh.warp_count[warp] = top;
            sh.warp_mass[warp] = low;
        }
        if (tid == 0) sh.list_size = 0u;
        __syncthreads();
        top = __reduce_max_sync(0xFFFFFFFFu, sh.warp_count[lane & 15]);
        low = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(sh.warp_mass[lane & 15]));
        u64 first = static_cast<u64>(top) << 32 | 0xFFFFFFFFu;   // no element's order is above it
        int shift = 56 - __clzll(first - (static_cast<u64>(low) << 32));
        uint32_t members;
        for (;;) {
            if (shift < 0) shift = 0;
            clear_bins();
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                if (!(in >> k & 1)) continue;
                const uint32_t b = static_cast<uint32_t>((first - order[k]) >> shift);
                atomicAdd(&sh.count[b], 1u);
                if (value[k] != 0) add_mass(&sh.mass[b], value[k]);
            }
            __syncthreads();
            const uint32_t c = tid < kBins ? sh.count[tid] : 0u;
            const u64 m = tid < kBins ? sh.mass[tid] : 0ull;
            u64 all;
            uint32_t all_c;
            const u64 before = block_before(m, sh.warp_mass, all);
            const uint32_t c0 = block_before(c, sh.warp_count, all_c);
            if (c != 0 && before < limit && (before + m >= limit || c0 + c == all_c))
                sh.decision = Decision{before, 0, 0, 0, static_cast<uint32_t>(tid), c};
            __syncthreads();
            const uint32_t bin = sh.decision.bin;
            limit -= sh.decision.mass;
            members = sh.decision.members;
#pragma unroll
            for (int k = 0; k < kEach; ++k)
                if (static_cast<uint32_t>((first - order[k]) >> shift) != bin) in &= ~(1u << k);
            if (members <= kFew) break;
            first -= static_cast<u64>(bin) << shift;
            shift -= 8;
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (!(in >> k & 1)) continue;
            const uint32_t at = atomicAdd(&sh.list_size, 1u);
            sh.few[at] = order[k];
            sh.few_value[at] = value[k];
        }
        __syncthreads();
        if (tid < members) {
            const u64 mine = sh.few[tid], v = sh.few_value[tid];
            uint32_t place = 0;
            u64 before = 0;
#pragma unroll 4
            for (uint32_t j = 0; j < members; ++j) {
                const bool earlier = sh.few[j] > mine;
                place += earlier ? 1u : 0u;
                before += earlier ? sh.few_value[j] : 0ull;
            }
            if (before < limit && (before + v >= limit || place == members - 1)) {
                sh.pick = mine;
                sh.pick_value = v;
            }
        }
        __syncthreads();
    }

    __device__ __forceinline__ void finish_parted(const SampleParams& p, int row, int n, int k, float top_p, float min_p,
                                                  u64 total) {
        u64 order[kEach], value[kEach], e[kEach], all = 0;
        float w[kEach];
        uint32_t in = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = threadIdx.x + j * kSampleThreads;
            if (i < n) in |= 1u << j;
            e[j] = i < n ? sh.list[i] : 0ull;
            w[j] = i < n ? weight(value_of(static_cast<uint32_t>(e[j] >> 32))) : 0.0f;
        }
        auto in_all = [&]() -> u64 {
            u64 own = 0, sum;
#pragma unroll
            for (int j = 0; j < kEach; ++j) own += in >> j & 1 ? mass(w[j]) : 0ull;
            (void)block_before(own, sh.warp_mass, sum);
            return sum;
        };
        // the first k, of those the ones that top_p keeps, and the draw among those in the order of their indices
#pragma unroll 1
        for (int stage = 0; stage < 3; ++stage) {
            u64 limit = static_cast<u64>(k);
            if (stage == 0 && k == n) continue;
            if (stage == 1) {
                if (!(top_p < 1.0f)) continue;
                if (total == 0) total = in_all();
                limit = by_one([&] { return mass_limit(top_p, total); });
            }
            if (stage == 2) {
#pragma unroll
                for (int j = 0; j < kEach; ++j)
                    if (w[j] < min_p || mass(w[j]) == 0) in &= ~(1u << j);
                all = in_all();
                limit = by_one([&] { return target_of(p.u[row], all); }) + 1;
            }
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                order[j] = stage == 2 ? e[j] << 32 : e[j];   // the lower half falls with the index
                value[j] = stage == 0 ? 1ull : mass(w[j]);
            }
            last_below(order, value, in, limit);
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if (order[j] < sh.pick) in &= ~(1u << j);
        }
        if (threadIdx.x == 0) {
            p.tokens[row] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(sh.pick >> 32));
            if (p.probs != nullptr) p.probs[row] = __fdiv_rn(static_cast<float>(sh.pick_value), static_cast<float>(all));
        }
    }

    __device__ __forceinline__ uint32_t block_total(uint32_t v) {
        v = __reduce_add_sync(0xFFFFFFFFu, v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh.warp_count[threadIdx.x >> 5] = v;
        __syncthreads();
        uint32_t all = 0;
        for (int w = 0; w < kSampleWarps; ++w) all += sh.warp_count[w];
        return all;
    }

    // ---- selection in general --------------------------------------------------------------------------------------

    __device__ __forceinline__ static float bins(float z) { return fminf(-z * kBinsPerUnit, static_cast<float>(kBins - 1)); }

    // Elements that the levels before `level` left over: same bin0, same bin1, same leading key bits.
    uint32_t bin0, bin1, prefix;
    __device__ __forceinline__ bool member(int level, float z, uint32_t key) const {
        if (level == 0) return true;
        const float t = bins(z);
        const uint32_t b = static_cast<uint32_t>(t);
        if (b != bin0) return false;
        if (level == 1) return true;
        if (sub_bin(t, b) != bin1) return false;
        return level == 2 || (key >> key_shift(level - 1)) == prefix;
    }
    __device__ __forceinline__ static uint32_t sub_bin(float t, uint32_t b) {
        // t - b is exact; the last bin is open and has no parts
        return b == kBins - 1 ? 0u : static_cast<uint32_t>((t - static_cast<float>(b)) * kBins);
    }
    __device__ __forceinline__ static int key_shift(int level) { return 8 * (5 - level); }
    __device__ __forceinline__ uint32_t digit(int level, float z, uint32_t key) const {
        if (level <= 1) {
            const float t = bins(z);
            const uint32_t b = static_cast<uint32_t>(t);
            return level == 0 ? b : sub_bin(t, b);
        }
        return kBins - 1 - ((key >> key_shift(level)) & (kBins - 1));   // the largest keys first
    }

    __device__ __forceinline__ void clear_bins() {
        if (threadIdx.x < kBins) {
            sh.count[threadIdx.x] = 0u;
            sh.mass[threadIdx.x] = 0ull;
        }
        __syncthreads();
    }

    // Joins the CTAs' histograms (every CTA does) and finds the bin of the last kept element: by count, rank < limit; by
    // mass, mass before < limit. The counts and masses before the histogram are given. With top_p_of_total the limit is that
    // share of the histogram's mass. The CTAs may still read one another's histograms when it returns.
    __device__ Decision join_bins(bool by_mass, u64 limit, u64 count_before, u64 mass_before, float top_p_of_total,
                                  bool with_mass = true) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        const int b = threadIdx.x;   // a bin for each of the first threads
        uint32_t c = 0;
        uint32_t all_c;
        u64 m = 0, all_m = 0, m0 = 0;
        if (b < kBins) {
#pragma unroll
            for (int h = 0; h < kRanks; h += 8) {
                if (h >= ranks) break;
                uint32_t rc[8];   // eight loads in flight at once
#pragma unroll
                for (int r = 0; r < 8; ++r) rc[r] = h + r < ranks ? cluster.map_shared_rank(&sh, h + r)->count[b] : 0u;
#pragma unroll
                for (int r = 0; r < 8; ++r) c += rc[r];
            }
        }
        if (with_mass) {
            if (b < kBins) {
#pragma unroll
                for (int h = 0; h < kRanks; h += 8) {
                    if (h >= ranks) break;
                    u64 rm[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) rm[r] = h + r < ranks ? cluster.map_shared_rank(&sh, h + r)->mass[b] : 0ull;
#pragma unroll
                    for (int r = 0; r < 8; ++r) m += rm[r];
                }
            }
            m0 = mass_before + block_before(m, sh.warp_mass, all_m);
            if (top_p_of_total > 0.0f) limit = by_one([&] { return mass_limit(top_p_of_total, all_m); });
        }
        const u64 c0 = count_before + block_before(c, sh.warp_count, all_c);
        if (threadIdx.x == 0) sh.decision.members = 0xFFFFFFFFu;   // none: everything lies above the threshold
        __syncthreads();
        const bool here = by_mass ? c != 0 && m0 < limit && m0 + m >= limit : c0 < limit && c0 + c >= limit;
        if (b < kBins && here) sh.decision = Decision{m0, all_m, limit, static_cast<uint32_t>(c0), static_cast<uint32_t>(b), c};
        __syncthreads();
        return sh.decision;
    }

    // The threshold among the members of one bin, collected in the first CTA's list: the last kept one.
    __device__ void threshold_of_list(int n, bool by_mass, u64 limit, const Decision& d) {
        if (rank == 0) {
            if (n <= kCounted) {
                const int tid = threadIdx.x;
                const u64 e = tid < n ? sh.list[tid] : 0ull;
                if (tid < kCounted) sh.mass[tid] = tid < n ? mass(weight(value_of(static_cast<uint32_t>(e >> 32)))) : 0ull;
                __syncthreads();
                uint32_t place = 0;
                u64 before = d.mass;
                if (tid < n) {
#pragma unroll 4
                    for (int j = 0; j < n; ++j) {
                        const bool first = sh.list[j] > e;
                        place += first ? 1u : 0u;
                        before += first ? sh.mass[j] : 0ull;
                    }
                }
                const bool keep = tid < n && (by_mass ? before < limit : d.count + static_cast<u64>(place) < limit);
                const uint32_t kept = block_total(keep ? 1u : 0u);
                if (keep && place == kept - 1) tell_threshold(e);
            } else {
                u64 order[kEach], value[kEach];
                uint32_t in = 0;
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    const int i = threadIdx.x + j * kSampleThreads;
                    if (i < n) in |= 1u << j;
                    order[j] = i < n ? sh.list[i] : 0ull;
                    value[j] = i >= n ? 0ull : by_mass ? mass(weight(value_of(static_cast<uint32_t>(order[j] >> 32)))) : 1ull;
                }
                last_below(order, value, in, limit - (by_mass ? d.mass : d.count));
                if (threadIdx.x == 0) tell_threshold(sh.pick);
            }
        }
        cg::this_cluster().sync();
        thr = sh.threshold;
    }
    __device__ __forceinline__ void tell_threshold(u64 e) {
        cg::cluster_group cluster = cg::this_cluster();
        for (int r = 0; r < ranks; ++r)
            cluster.map_shared_rank(&sh, r)->threshold =
                Threshold{static_cast<uint32_t>(e >> 32), 0xFFFFFFFFu - static_cast<uint32_t>(e)};
    }
    // Lower the threshold to the last element kept by the rank limit (by count) or by top_p (by mass).
    __device__ void select(bool by_mass, u64 limit, float top_p) {
        cg::cluster_group cluster = cg::this_cluster();
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        Decision d{0, 0, 0, 0, 0, 0};
        bin0 = bin1 = prefix = 0;
        int level = 0;
        for (;;) {
            cluster.sync();   // no CTA reads another's histogram any more
            clear_bins();
            for (int i = lo + tid; i < hi; i += kSampleThreads) {
                const float l = slot(i);
                const uint32_t key = key_of(l);
                if (!under(key, index(i))) continue;
                const float z = depth(l);
                if (!member(level, z, key)) continue;
                const uint32_t b = digit(level, z, key);
                atomicAdd(&sh.count[b], 1u);
                const u64 m = mass(weight(l, z));
                if (m != 0) add_mass(&sh.mass[b], m);
            }
            d = join_bins(by_mass, limit, d.count, d.mass, level == 0 ? top_p : 0.0f);
            if (level == 0 && by_mass) limit = d.limit;
            if (level == 0) bin0 = d.bin;
            if (level == 1) bin1 = d.bin;
            if (level >= 2) {
                const uint32_t dig = kBins - 1 - d.bin;
                prefix = level == 2 ? dig : prefix << 8 | dig;
            }
            ++level;
            if (d.members <= kList || level == 6) break;
        }
        if (d.members <= kList) {
            __syncthreads();
            clear_list();
            cluster.sync();   // the first CTA's list is free
            for (int i = lo + tid; i < hi; i += kSampleThreads) {
                const float l = slot(i);
                const uint32_t key = key_of(l);
                if (under(key, index(i)) && member(level, depth(l), key)) add(key, index(i));
            }
            const int n = collect();
            if (n <= kList) {
                threshold_of_list(n, by_mass, limit, d);
                return;
            }
            // all members in the part of one CTA: on to single logits
            for (; level < 6; ++level) {
                cluster.sync();
                clear_bins();
                for (int i = lo + tid; i < hi; i += kSampleThreads) {
                    const float l = slot(i);
                    const uint32_t key = key_of(l);
                    const float z = depth(l);
                    if (!under(key, index(i)) || !member(level, z, key)) continue;
                    atomicAdd(&sh.count[digit(level, z, key)], 1u);
                    add_mass(&sh.mass[digit(level, z, key)], mass(weight(l, z)));
                }
                d = join_bins(by_mass, limit, d.count, d.mass, 0.0f);
                if (level == 1) bin1 = d.bin;
                if (level >= 2) {
                    const uint32_t dig = kBins - 1 - d.bin;
                    prefix = level == 2 ? dig : prefix << 8 | dig;
                }
            }
        }
        // equal logits, more than the list holds: the first `keep` of them by index
        const uint32_t key = prefix;
        const u64 m = mass(weight(value_of(key)));
        u64 keep = d.members;
        if (by_mass) {
            u64 a = 0, b = d.members;   // the first i whose mass before is not below the limit
            while (a < b) {
                const u64 mid = (a + b) / 2;
                if (d.mass + mid * m < limit) a = mid + 1;
                else b = mid;
            }
            keep = a;
        } else {
            keep = limit - d.count;
        }
        const int seg = ((hi - lo + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32;
        const int s0 = lo + warp * seg, s1 = s0 + seg < hi ? s0 + seg : hi;
        uint32_t equal = 0;
        for (int i = s0 + lane; i < s1; i += 32) {
            const uint32_t k2 = key_of(slot(i));
            equal += k2 == key && under(k2, index(i)) ? 1u : 0u;
        }
        equal = __reduce_add_sync(0xFFFFFFFFu, equal);
        if (lane == 0) sh.warp_count[warp] = equal;
        __syncthreads();
        u64 mine = 0, at = 0;
        for (int w = 0; w < kSampleWarps; ++w) {
            if (w < warp) at += sh.warp_count[w];
            mine += sh.warp_count[w];
        }
        if (tid < ranks) cluster.map_shared_rank(&sh, tid)->sum[rank] = mine;
        cluster.sync();
        for (int r = 0; r < rank; ++r) at += sh.sum[r];
        if (at < keep && at + equal >= keep) {
            for (int i0 = s0; i0 < s1; i0 += 32) {
                const int i = i0 + lane;
                const bool in = i < s1 && key_of(slot(i)) == key && under(key, index(i));
                const uint32_t votes = __ballot_sync(0xFFFFFFFFu, in);
                const u64 place = at + __popc(votes & ((1u << lane) - 1u));
                if (in && place == keep - 1) {
                    const Threshold t{key, index(i)};
                    for (int r = 0; r < ranks; ++r) cluster.map_shared_rank(&sh, r)->threshold = t;
                }
                at += __popc(votes);
            }
        }
        cluster.sync();
        thr = sh.threshold;
    }
};

template <class T, bool HELD>
__global__ void __launch_bounds__(kSampleThreads, 2) qmm_sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(16) float slots[];
    __shared__ SampleShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int kRead = 16 / sizeof(T);
    constexpr int kVec = RowSampler<T, HELD>::kVec;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / ranks;
    auto started = cluster.barrier_arrive();   // waited for before the first access to another CTA's memory
    griddep_launch_dependents();
    griddep_wait();

    // this CTA's 16-byte chunks of the row; slot 0 is the first element of its first chunk
    const T* src = static_cast<const T*>(p.logits) + row * p.stride;
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    const int reads = (lead + p.vocab + kRead - 1) / kRead;
    const int reads_here = (reads + ranks - 1) / ranks, per_cta = reads_here * (kRead / kVec);   // per_cta: chunks
    RowSampler<T, HELD> s{sh, slots, src};
    s.chunks = per_cta;
    s.shift = rank * reads_here * kRead - lead;
    const int left = p.vocab - s.shift;
    s.lo = s.shift < 0 ? -s.shift : 0;
    s.hi = left < per_cta * kVec ? (left > s.lo ? left : s.lo) : per_cta * kVec;
    s.rank = rank;
    s.ranks = ranks;
    s.temperature = p.temperature[row];
    const int top_k = p.top_k[row];
    const float top_p = p.top_p[row], min_p = p.min_p[row];

    // every thread's largest logit, and the logits to shared memory
    float best = -INFINITY;
    RowSampler<T, false>{sh, nullptr, src, s.lo, s.hi, reads_here, s.shift}.each_chunk(
        tid, reads_here, kSampleThreads, [&](int c, const float(&v)[kRead]) {
#pragma unroll
            for (int e = 0; e < kRead; ++e) best = fmaxf(best, v[e]);
            if constexpr (HELD) {
#pragma unroll
                for (int e = 0; e < kRead; e += 4)
                    *reinterpret_cast<float4*>(slots + c * kRead + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
        });
    // The row's largest logit, and the mean of the threads' largest ones (those of numbers in use, not of masks).
    {
        const uint32_t key = __reduce_max_sync(0xFFFFFFFFu, key_of(best));
        const bool in_use = best > -1e30f && best < 1e30f;
        const float sum = warp_add(in_use ? best : 0.0f);
        const uint32_t some = __popc(__ballot_sync(0xFFFFFFFFu, in_use));
        if (lane == 0) {
            sh.warp_count[warp] = key;
            sh.warp_mass[warp] = static_cast<u64>(__float_as_uint(sum)) << 32 | some;
        }
        __syncthreads();
        cluster.barrier_wait(std::move(started));
        if (tid < ranks) {
            uint32_t k = 0, n = 0;
            float f = 0.0f;
            for (int w = 0; w < kSampleWarps; ++w) {
                k = sh.warp_count[w] > k ? sh.warp_count[w] : k;
                f += __uint_as_float(static_cast<uint32_t>(sh.warp_mass[w] >> 32));
                n += static_cast<uint32_t>(sh.warp_mass[w]);
            }
            SampleShared* o = cluster.map_shared_rank(&sh, tid);
            o->top[rank] = value_of(k);
            o->level[rank] = f;
            o->above[rank] = static_cast<float>(n);
        }
    }
    if (tid < kBins) {
        sh.count[tid] = 0u;
        sh.mass[tid] = 0ull;
    }
    s.clear_list();
    cluster.sync();
    float level, above;
    {
        const bool in = lane < ranks;
        s.top = value_of(__reduce_max_sync(0xFFFFFFFFu, in ? key_of(sh.top[lane]) : 0u));
        level = warp_add(in ? sh.level[lane] : 0.0f);
        above = warp_add(in ? sh.above[lane] : 0.0f);
    }
    s.thr = Threshold{0u, 0xFFFFFFFFu};
    if (s.top == -INFINITY) {
        if (rank == 0 && tid == 0) {
            p.tokens[row] = -1;
            if (p.probs != nullptr) p.probs[row] = 0.0f;
        }
        return;
    }

    const bool by_count = top_k > 0 && top_k < p.vocab;
    const bool by_mass = top_p < 1.0f;
    if (!(s.temperature > 0.0f) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {
        // the first of the largest
        uint32_t first = 0xFFFFFFFFu;
        s.each_chunk_of(best == s.top, [&](int c, const float(&v)[kVec]) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (v[e] == s.top) first = min(first, s.index(c * kVec + e));
        });
        first = __reduce_min_sync(0xFFFFFFFFu, first);
        if (lane == 0) sh.warp_count[warp] = first;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kSampleWarps; ++w) first = min(first, sh.warp_count[w]);
            cluster.map_shared_rank(&sh, 0)->sum[rank] = first;
        }
        cluster.sync();
        if (rank == 0 && tid == 0) {
            for (int r = 0; r < ranks; ++r) first = min(first, static_cast<uint32_t>(sh.sum[r]));
            p.tokens[row] = static_cast<int32_t>(first);
            if (p.probs != nullptr) p.probs[row] = 1.0f;
        }
        return;
    }

    if (by_count && top_k <= kList / 2 && s.top < 1e30f) {
        // The bin of the k-th of the threads' largest logits, or of the chunks' largest ones where k is a large part of the
        // threads, or of all logits.
        const bool of_threads = top_k <= ranks * kSampleThreads / 4, of_chunks = top_k <= reads / 4;
        const float range = above > 0.0f ? (of_threads ? 1.5f : of_chunks ? 2.5f : 4.0f) * (s.top - level / above) : 0.0f;
        const float per_unit = range > 0.0f ? kBins / range : 1.0f;
        auto bin_of = [&](float l) -> int { return static_cast<int>(fminf((s.top - l) * per_unit, kBins - 1.0f)); };
        if (of_threads) {
            if (best > -INFINITY) atomicAdd(&sh.count[bin_of(best)], 1u);
        } else {
            s.each_chunk(tid, per_cta, kSampleThreads, [&](int c, const float(&v)[kVec]) {
                float l = v[0];
#pragma unroll
                for (int e = 1; e < kVec; ++e) l = fmaxf(l, v[e]);
                if (of_chunks) {
                    if (l > -INFINITY) atomicAdd(&sh.count[bin_of(l)], 1u);
                } else {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (v[e] > -INFINITY) atomicAdd(&sh.count[bin_of(v[e])], 1u);
                }
            });
        }
        const Decision d = s.join_bins(false, static_cast<u64>(top_k), 0, 0, 0.0f, false);
        if (d.members != 0xFFFFFFFFu && d.bin < kBins - 1) {
            const float below = static_cast<float>(d.bin + 1);
            auto add_above = [&](int c, const float(&v)[kVec]) {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if ((s.top - v[e]) * per_unit < below) s.add(key_of(v[e]), s.index(c * kVec + e));
            };
            if (of_threads) s.each_chunk_of((s.top - best) * per_unit < below, add_above);
            else s.each_chunk(tid, per_cta, kSampleThreads, add_above);
            const int n = s.collect();
            if (n <= kList) {
                if (rank == 0) s.finish(p, row, n, top_k, top_p, min_p, 0);
                return;
            }
        }
    }

    // The weights (HELD: in the logits' place), and a histogram of their masses or their sums by warps, which have segments
    // of the row.
    const int seg = (per_cta + kSampleWarps - 1) / kSampleWarps;
    const int s0 = warp * seg, s1 = s0 + seg < per_cta ? s0 + seg : per_cta;   // in chunks
    bool general = by_count;     // thresholds by logit and index, the logits still in their place
    u64 own = 0;
    uint32_t edge = 0;           // HELD: weights of fewer bits lie in bins after the threshold's
    auto bits_below = [](float w) -> uint32_t { return 0x3F800000u - __float_as_uint(w); };
    auto bin_of = [&](float w) -> uint32_t { return min(bits_below(w) >> kWeightBinShift, static_cast<uint32_t>(kBins - 1)); };
    if (!general) {
        __syncthreads();
        s.each_chunk(s0 + lane, s1, 32, [&](int c, const float(&v)[kVec]) {
            float w[kVec];
            s.weights(v, w);
            u64 m[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                m[e] = s.mass(w[e]);
                w[e] = m[e] != 0 ? w[e] : 0.0f;
            }
            if (by_mass) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    if (m[e] == 0) continue;
                    atomicAdd(&sh.count[bin_of(w[e])], 1u);
                    add_mass(&sh.mass[bin_of(w[e])], m[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) own += w[e] < min_p ? 0 : m[e];
            }
            if constexpr (HELD) {
                *reinterpret_cast<float4*>(slots + c * kVec) = make_float4(w[0], w[1], w[2], w[3]);
            }
        });
    }
    // f(i, w) for the slots whose weights have bits_below in [from, to]. Unless they are HELD, a range of logits a little wider
    // (by the rounding of all between logit and weight) says which weights to look at.
    auto each_between = [&](uint32_t from, uint32_t to, auto f) {
        float low = __uint_as_float(0x3F800000u - to), high = __uint_as_float(0x3F800000u - from);
        if constexpr (!HELD) {
            const float slack = fabsf(s.top) * 2.5e-7f;
            low = fmaf(logf(low) - 1e-3f, s.temperature, s.top) - slack;
            high = fmaf(logf(high) + 1e-3f, s.temperature, s.top) + slack;
        }
        s.each_chunk(tid, per_cta, kSampleThreads, [&](int c, const float(&v)[kVec]) {
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < kVec; ++e) hits |= v[e] < low || v[e] > high ? 0u : 1u << e;   // all if no numbers
            for (; hits != 0; hits &= hits - 1) {
                const int e = __ffs(hits) - 1, i = c * kVec + e;
                float w = s.pick(v, e);
                if constexpr (!HELD) w = s.weight(w);
                if (w > 0.0f && s.mass(w) != 0 && bits_below(w) - from <= to - from) f(i, w);
            }
        });
    };
    if (!general && by_mass) {
        Decision d = s.join_bins(true, 0, 0, 0, top_p);
        const u64 total = d.total, limit = d.limit;
        general = d.members == 0xFFFFFFFFu || d.bin == kBins - 1;
        const bool whole = !general && d.count + d.members <= kCounted;   // few in all: the draw is the first CTA's
        const uint32_t bin = d.bin;
        uint32_t sub = 0xFFFFFFFFu;                                       // part of the bin
        constexpr int kSubShift = kWeightBinShift - 8;
        if (!general && !whole && d.members > kCounted) {
            // the next bits part the bin's members
            cluster.sync();
            s.clear_bins();
            each_between(bin << kWeightBinShift, (bin + 1 << kWeightBinShift) - 1, [&](int, float w) {
                const uint32_t b = bits_below(w) >> kSubShift & (kBins - 1);
                atomicAdd(&sh.count[b], 1u);
                add_mass(&sh.mass[b], s.mass(w));
            });
            d = s.join_bins(true, limit, d.count, d.mass, 0.0f);
            sub = d.bin;
            general = d.members == 0xFFFFFFFFu || d.members > kList;
        }
        if (!general) {
            const bool parted = sub != 0xFFFFFFFFu;
            const uint32_t from = (bin << kWeightBinShift) + (parted ? sub << kSubShift : 0u);
            const uint32_t past = from + (1u << (parted ? kSubShift : kWeightBinShift));
            // their slots first: the logits come from memory again, all at once
            each_between(whole ? 0u : from, past - 1, [&](int i, float) {
                const uint32_t at = atomicAdd(&sh.list_size, 1u);
                if (at < kList) sh.own[at] = static_cast<uint32_t>(i);
            });
            __syncthreads();
            const int mine = static_cast<int>(min(sh.list_size, static_cast<uint32_t>(kList / ranks)));
            for (int k = tid; k < mine; k += kSampleThreads) {
                const uint32_t index = s.index(sh.own[k]);
                cluster.map_shared_rank(&sh, 0)->list[rank * (kList / ranks) + k] = entry_of(key_of(s.logit_at(index)), index);
            }
            const int n = s.collect();
            if (n > kList) {
                general = true;
            } else if (whole) {
                if (rank == 0) s.finish(p, row, n, 0, top_p, min_p, total);
                return;
            } else {
                s.threshold_of_list(n, true, limit, d);
                if constexpr (HELD) {   // members past the threshold lose their weight
                    for (int k = tid; k < mine; k += kSampleThreads) {
                        const uint32_t index = s.index(sh.own[k]);
                        if (!s.under(key_of(s.logit_at(index)), index)) slots[sh.own[k]] = 0.0f;
                    }
                    __syncthreads();
                    edge = 0x3F800000u - past + 1;
                }
            }
        }
        if (HELD && general) {   // the logits again
            __syncthreads();
            for (int i = tid; i < per_cta * kVec; i += kSampleThreads)
                slots[i] = i >= s.lo && i < s.hi ? s.logit_at(s.index(i)) : -INFINITY;
            __syncthreads();
        }
    }
    if (general) {
        if (by_count) s.select(false, static_cast<u64>(top_k), 0.0f);
        if (by_mass) s.select(true, 0, top_p);
    }

    // the draw: kept masses in the order of the indices
    const bool by_logit = !HELD || general;
    auto kept = [&](int i, float v) -> u64 {
        if (by_logit) {
            if (!s.under(key_of(v), s.index(i))) return 0;
            v = s.weight(v);
        } else if (__float_as_uint(v) < edge) {
            return 0;
        }
        return v < min_p ? 0 : s.mass(v);
    };
    auto kept_of = [&](int c, const float(&v)[kVec]) -> u64 {
        u64 sum = 0;
        if (by_logit) {
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < kVec; ++e) hits |= v[e] > -INFINITY && s.under(key_of(v[e]), s.index(c * kVec + e)) ? 1u << e : 0u;
            for (; hits != 0; hits &= hits - 1) {
                const int e = __ffs(hits) - 1;
                sum += kept(c * kVec + e, s.pick(v, e));
            }
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) sum += v[e] < min_p || __float_as_uint(v[e]) < edge ? 0ull : s.mass(v[e]);
        }
        return sum;
    };
    if (general || by_mass) {
        own = 0;
        s.each_chunk(s0 + lane, s1, 32, [&](int c, const float(&v)[kVec]) { own += kept_of(c, v); });
    }
    own = warp_add(own);
    __syncthreads();
    if (lane == 0) sh.warp_mass[warp] = own;
    __syncthreads();
    u64 before = 0, all = 0;
    for (int w = 0; w < kSampleWarps; ++w) {
        if (w < warp) before += sh.warp_mass[w];
        all += sh.warp_mass[w];
    }
    if (tid < ranks) cluster.map_shared_rank(&sh, tid)->sum[rank] = all;
    cluster.sync();
    u64 total = 0, before_cta = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r < rank) before_cta += sh.sum[r];
        total += sh.sum[r];
    }
    before += before_cta;
    const u64 target = s.by_one([&] { return s.target_of(p.u[row], total); });
    if (target < before_cta || target >= before_cta + all) return;
    int c0 = s0, c1 = s1;
    if (seg > 4 * 32) {   // all warps part the segment of the one that has it
        if (lane == 0 && target >= before && target < before + own) {
            sh.pick = before;
            sh.decision.bin = static_cast<uint32_t>(warp);
        }
        __syncthreads();
        const int first = static_cast<int>(sh.decision.bin) * seg, part = (seg + kSampleWarps - 1) / kSampleWarps;
        const int end = first + seg < per_cta ? first + seg : per_cta;
        c0 = first + warp * part;
        c1 = c0 + part < end ? c0 + part : end;
        own = 0;
        s.each_chunk(c0 + lane, c1, 32, [&](int c, const float(&v)[kVec]) { own += kept_of(c, v); });
        own = warp_add(own);
        if (lane == 0) sh.warp_mass[warp] = own;
        __syncthreads();
        before = sh.pick;
        for (int w = 0; w < warp; ++w) before += sh.warp_mass[w];
    }
    if (target < before || target >= before + own) return;
    for (; c0 < c1; c0 += 32) {
        const int c = c0 + lane;
        u64 sum = 0;
        if (c < c1) {
            float v[kVec];
            s.load(c, v);
            sum = kept_of(c, v);
        }
        u64 upto = before + warp_scan(sum, lane);
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > target);
        if (past != 0) {
            if (lane == __ffs(past) - 1) {
                upto -= sum;
                int i = c * kVec;
                u64 m = kept(i, s.slot(i));
                while (upto + m <= target && i < c * kVec + kVec - 1) {
                    upto += m;
                    ++i;
                    m = kept(i, s.slot(i));
                }
                p.tokens[row] = static_cast<int32_t>(s.index(i));
                if (p.probs != nullptr) p.probs[row] = __fdiv_rn(static_cast<float>(m), static_cast<float>(total));
            }
            return;
        }
        before = __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
}

// A CTA's share of a row in shared memory: at most this many bytes.
constexpr int kSampleSmem = 4 * 8 * ((QMM_SAMPLE_MAX_VOCAB / 8 + 1 + kPortableRanks - 1) / kPortableRanks);
static_assert(kSampleSmem + sizeof(SampleShared) <= 227 * 1024, "the largest row fits its cluster");

template <class T, bool HELD>
int launch(const SampleParams& p, int M, int ranks, cudaStream_t stream) {
    if (HELD) {
        static std::atomic<u64> configured{0};   // one bit for each device
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return QMM_ERR_CUDA;
        if (dev >= 64 || !(configured.load(std::memory_order_relaxed) >> dev & 1)) {
            const void* kernel = reinterpret_cast<const void*>(&qmm_sample_kernel<T, HELD>);
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSampleSmem) != cudaSuccess ||
                cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
                return QMM_ERR_CUDA;
            if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_relaxed);
        }
    }
    while (ranks > 1 && p.vocab / ranks < 2048) ranks /= 2;   // shorter shares cost more exchange than they save
    const int vec = 16 / static_cast<int>(sizeof(T));
    const int chunks = (p.vocab + vec - 1) / vec + 1;         // one more where the row starts inside a chunk
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(M) * ranks);
    cfg.blockDim = dim3(kSampleThreads);
    cfg.dynamicSmemBytes = HELD ? static_cast<size_t>((chunks + ranks - 1) / ranks) * vec * 4 : 0;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, qmm_sample_kernel<T, HELD>, p) == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

// Few rows are split over many CTAs, which keep them. Where those would not all fit the GPU at once, as few CTAs a row as
// fill it read the row again from the L2 cache when they need it: their exchanges cost less, and none waits for others.
template <class T>
int launch_rows(const SampleParams& p, int M, cudaStream_t stream) {
    if (M * kPortableRanks <= kManyCtas) return launch<T, true>(p, M, M <= 8 ? kRanks : kPortableRanks, stream);
    int ranks = kPortableRanks / 2;
    while (ranks > 1 && M * ranks > kManyCtas) ranks /= 2;
    return launch<T, false>(p, M, ranks, stream);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

}  // namespace qmmk

extern "C" int qmm_sample(const void* logits, int M, int vocab, int64_t stride, int in_dtype, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                          int32_t* tokens, float* probs, void* stream) {
    using namespace qmmk;
    if (in_dtype != QMM_IN_F32 && in_dtype != QMM_IN_BF16) return QMM_ERR_INVALID_ARG;
    if (M < 0 || M > (1 << 24) || vocab < 1) return QMM_ERR_INVALID_ARG;
    if (vocab > QMM_SAMPLE_MAX_VOCAB) return QMM_ERR_UNSUPPORTED;
    if (M == 0) return QMM_OK;
    if (M > 1 && (stride < vocab || stride > (1LL << 40))) return QMM_ERR_INVALID_ARG;
    if (logits == nullptr || !aligned(logits, in_dtype == QMM_IN_F32 ? 4 : 2)) return QMM_ERR_INVALID_ARG;
    const void* rows[6] = {temperature, top_k, top_p, min_p, u, tokens};
    for (const void* r : rows)
        if (r == nullptr || !aligned(r, 4)) return QMM_ERR_INVALID_ARG;
    if (!aligned(probs, 4)) return QMM_ERR_INVALID_ARG;
    SampleParams sp;
    sp.logits = logits;
    sp.stride = stride;
    sp.temperature = temperature;
    sp.top_k = top_k;
    sp.top_p = top_p;
    sp.min_p = min_p;
    sp.u = u;
    sp.tokens = tokens;
    sp.probs = probs;
    sp.vocab = vocab;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return in_dtype == QMM_IN_F32 ? launch_rows<float>(sp, M, st) : launch_rows<uint16_t>(sp, M, st);
}
