// Draw of the next token from logits: temperature, top-k, top-p, min-p.
//
//   w_i = exp((l_i - max l) / T) held as the whole number floor(2^40 w_i);
//   kept: rank < top_k, mass before < top_p * mass of the top_k, w_i >= min_p;
//   token: the first index whose sum of kept mass exceeds floor(u * kept mass).
//
// Whole-number masses add up to the same sum in any order (a row holds less
// than 2^59), so histograms with atomics, any split of the row and any order of
// arrival give the same token.
//
// A row is one cluster's: its CTAs read it once from memory, keep it in shared
// memory and exchange maxima, histograms and sums through distributed shared
// memory. top-k and top-p are thresholds in the order (logit falling, index
// rising). One histogram of count and mass over (max l - l) / T finds the bin
// that a threshold lies in; its few members are then ranked against one
// another. Only where a bin holds too many are they parted further: by the next
// bits of the same distance, then by the bits of the logit, last by index.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>

#include "../../include/qmm.h"
#include "qmm_device.cuh"

namespace qmmk {

namespace {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 1024;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kBins = kSampleThreads;      // one thread of the first CTA joins one bin
constexpr int kCap = 1024;                 // members of a bin that are ranked one by one
constexpr int kMaxCluster = 8;
constexpr float kWeightOne = 1099511627776.0f;   // 2^40
constexpr float kBinsPerUnit = 32.0f;      // bins for one unit of (max l - l) / T: mass ends at 27.7 units

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
    uint32_t count;  // elements ranked before the bin
    uint32_t bin;
    uint32_t members;
};

struct Threshold {   // kept: key > key, or key == key and index <= index
    uint32_t key;
    uint32_t index;
};

struct SampleShared {
    u64 best[kMaxCluster];
    u64 sum[kMaxCluster];
    u64 warp_mass[kSampleWarps];
    u64 mass[kBins];
    uint32_t count[kBins];
    uint32_t warp_count[kSampleWarps];
    uint32_t list_key[kCap];
    uint32_t list_index[kCap];
    u64 list_mass[kCap];
    uint32_t list_size;
    Decision decision;
    Threshold threshold;
};

// Unsigned numbers in the order of the floats; NaN is -infinity, and -0 is 0.
__device__ __forceinline__ float clean(float l) { return l != l ? -INFINITY : l + 0.0f; }
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
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

template <class T>
struct RowSampler {
    SampleShared& sh;
    const T* x;            // this CTA's slots
    int lo, hi;            // the slots that hold logits
    int64_t shift;         // index of slot 0
    int rank, ranks;
    float top, temperature;
    Threshold thr;

    __device__ __forceinline__ float logit(int i) const {
        if constexpr (sizeof(T) == 2)
            return clean(__uint_as_float(static_cast<uint32_t>(x[i]) << 16));
        else
            return clean(x[i]);
    }
    __device__ __forceinline__ uint32_t index(int i) const { return static_cast<uint32_t>(shift + i); }
    __device__ __forceinline__ float depth(float l) const { return l == top ? 0.0f : __fdiv_rn(l - top, temperature); }
    __device__ __forceinline__ float weight(float l, float z) const { return l == top ? 1.0f : expf(z); }
    // (not above 0 also where an infinite temperature or logit leaves no number)
    __device__ __forceinline__ u64 mass(float w) const { return w > 0.0f ? static_cast<u64>(w * kWeightOne) : 0ull; }
    __device__ __forceinline__ bool under(uint32_t key, uint32_t idx) const {
        return key > thr.key || (key == thr.key && idx <= thr.index);
    }
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
    __device__ __forceinline__ static int key_shift(int level) { return level == 2 ? 22 : level == 3 ? 12 : level == 4 ? 2 : 0; }
    __device__ __forceinline__ uint32_t digit(int level, float z, uint32_t key) const {
        if (level <= 1) {
            const float t = bins(z);
            const uint32_t b = static_cast<uint32_t>(t);
            return level == 0 ? b : sub_bin(t, b);
        }
        return kBins - 1 - ((key >> key_shift(level)) & (kBins - 1));   // the largest keys first
    }

    // One level: which bin holds the last kept element. By count: rank < limit. By mass: mass before < limit.
    __device__ Decision level_pass(int level, bool by_mass, u64 limit_count, float top_p, double limit_mass,
                                   u64 count_before, u64 mass_before) {
        cg::cluster_group cluster = cg::this_cluster();
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        sh.count[tid] = 0u;
        sh.mass[tid] = 0ull;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += kSampleThreads) {
            const float l = logit(i);
            const uint32_t key = key_of(l);
            if (!under(key, index(i))) continue;
            const float z = depth(l);
            if (!member(level, z, key)) continue;
            const uint32_t d = digit(level, z, key);
            atomicAdd(&sh.count[d], 1u);
            const u64 m = mass(weight(l, z));
            if (m != 0) atomicAdd(&sh.mass[d], m);
        }
        cluster.sync();
        if (rank == 0) {
            u64 c = 0, m = 0;
            for (int r = 0; r < ranks; ++r) {
                const SampleShared* o = cluster.map_shared_rank(&sh, r);
                c += o->count[tid];
                m += o->mass[tid];
            }
            const u64 c_in = warp_scan(c, lane), m_in = warp_scan(m, lane);
            if (lane == 31) {
                sh.warp_count[warp] = static_cast<uint32_t>(c_in);
                sh.warp_mass[warp] = m_in;
            }
            __syncthreads();
            u64 c_off = count_before, m_off = mass_before, total = 0;
            for (int w = 0; w < kSampleWarps; ++w) {
                if (w < warp) c_off += sh.warp_count[w], m_off += sh.warp_mass[w];
                total += sh.warp_mass[w];
            }
            const u64 c1 = c_off + c_in, m1 = m_off + m_in, c0 = c1 - c, m0 = m1 - m;
            bool here;
            if (by_mass) {
                const double limit = level == 0 ? static_cast<double>(top_p) * static_cast<double>(total) : limit_mass;
                here = c != 0 && static_cast<double>(m0) < limit && !(static_cast<double>(m1) < limit);
            } else {
                here = c0 < limit_count && c1 >= limit_count;
            }
            if (here) {
                const Decision d{m0, total, static_cast<uint32_t>(c0), static_cast<uint32_t>(tid), static_cast<uint32_t>(c)};
                for (int r = 0; r < ranks; ++r) cluster.map_shared_rank(&sh, r)->decision = d;
            }
        }
        cluster.sync();
        return sh.decision;
    }

    // Lower the threshold to the last element kept by the rank limit (by count) or by top_p (by mass).
    __device__ void select(bool by_mass, u64 limit_count, float top_p) {
        cg::cluster_group cluster = cg::this_cluster();
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        double limit = 0.0;
        Decision d{0, 0, 0, 0, 0};
        bin0 = bin1 = prefix = 0;
        int level = 0;
        for (;;) {
            d = level_pass(level, by_mass, limit_count, top_p, limit, d.count, d.mass);
            if (level == 0) limit = static_cast<double>(top_p) * static_cast<double>(d.total);
            if (level == 0) bin0 = d.bin;
            if (level == 1) bin1 = d.bin;
            if (level >= 2) {
                const uint32_t dig = kBins - 1 - d.bin;
                prefix = level == 2 ? dig : level == 5 ? (prefix << 2) | dig : (prefix << 10) | dig;
            }
            ++level;
            if (d.members <= kCap || level == 6) break;
        }
        if (d.members <= kCap) {
            // rank the members against one another in the first CTA
            SampleShared* first = cluster.map_shared_rank(&sh, 0);
            if (rank == 0 && tid == 0) sh.list_size = 0u;
            cluster.sync();
            for (int i = lo + tid; i < hi; i += kSampleThreads) {
                const float l = logit(i);
                const uint32_t key = key_of(l);
                if (!under(key, index(i))) continue;
                const float z = depth(l);
                if (!member(level, z, key)) continue;
                const uint32_t at = atomicAdd(&first->list_size, 1u);
                if (at < kCap) {
                    first->list_key[at] = key;
                    first->list_index[at] = index(i);
                    first->list_mass[at] = mass(weight(l, z));
                }
            }
            cluster.sync();
            if (rank == 0) {
                const int n = static_cast<int>(d.members);
                bool kept = false;
                u64 before = d.mass;
                uint32_t place = 0, key = 0, idx = 0;
                if (tid < n) {
                    key = sh.list_key[tid];
                    idx = sh.list_index[tid];
                    for (int j = 0; j < n; ++j) {
                        const uint32_t k2 = sh.list_key[j], i2 = sh.list_index[j];
                        if (k2 > key || (k2 == key && i2 < idx)) {
                            ++place;
                            before += sh.list_mass[j];
                        }
                    }
                    kept = by_mass ? static_cast<double>(before) < limit : d.count + place < limit_count;
                }
                const int keep = __syncthreads_count(kept);
                if (kept && place == static_cast<uint32_t>(keep - 1)) {
                    const Threshold t{key, idx};
                    for (int r = 0; r < ranks; ++r) cluster.map_shared_rank(&sh, r)->threshold = t;
                }
            }
            cluster.sync();
            thr = sh.threshold;
            return;
        }
        // more equal logits than the list holds: the first `keep` of them by index
        const uint32_t key = prefix;
        const float l0 = value_of(key);
        const u64 m = mass(weight(l0, depth(l0)));
        u64 keep = d.members;
        if (by_mass) {
            u64 a = 0, b = d.members;   // the first i whose mass before is not below the limit
            while (a < b) {
                const u64 mid = (a + b) / 2;
                if (static_cast<double>(d.mass + mid * m) < limit) a = mid + 1;
                else b = mid;
            }
            keep = a;
        } else {
            keep = limit_count - d.count;
        }
        const int seg = ((hi - lo + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32;
        const int s0 = lo + warp * seg, s1 = s0 + seg < hi ? s0 + seg : hi;
        uint32_t equal = 0;
        for (int i = s0 + lane; i < s1; i += 32) {
            const uint32_t k2 = key_of(logit(i));
            equal += k2 == key && under(k2, index(i)) ? 1u : 0u;
        }
        equal = warp_add(equal);
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
                const bool in = i < s1 && key_of(logit(i)) == key && under(key, index(i));
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

template <class T>
__global__ void __launch_bounds__(kSampleThreads) qmm_sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(16) uint8_t slots[];
    __shared__ SampleShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int kVec = 16 / sizeof(T);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / ranks;
    griddep_launch_dependents();
    griddep_wait();

    // this CTA's 16-byte chunks of the row; slot 0 is the first element of its first chunk
    const T* src = static_cast<const T*>(p.logits) + row * p.stride;
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    const int chunks = (lead + p.vocab + kVec - 1) / kVec;
    const int per_cta = (chunks + ranks - 1) / ranks;
    const int64_t shift = static_cast<int64_t>(rank) * per_cta * kVec - lead;   // index of slot 0
    const int64_t left = p.vocab - shift;
    T* const x = reinterpret_cast<T*>(slots);
    RowSampler<T> s{sh, x};
    s.shift = shift;
    s.lo = shift < 0 ? static_cast<int>(-shift) : 0;
    s.hi = left < per_cta * kVec ? (left > s.lo ? static_cast<int>(left) : s.lo) : per_cta * kVec;
    s.rank = rank;
    s.ranks = ranks;

    u64 best = 0;
    for (int c = tid; c < per_cta; c += kSampleThreads) {
        const int at = c * kVec;
        if (at >= s.lo && at + kVec <= s.hi) {
            *reinterpret_cast<uint4*>(x + at) = __ldg(reinterpret_cast<const uint4*>(src + shift + at));
        } else {
            for (int j = at; j < at + kVec; ++j)
                if (j >= s.lo && j < s.hi) x[j] = src[shift + j];
        }
        for (int j = at; j < at + kVec; ++j) {
            if (j < s.lo || j >= s.hi) continue;
            const u64 v = static_cast<u64>(key_of(s.logit(j))) << 32 | (0xFFFFFFFFu - s.index(j));
            best = v > best ? v : best;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 v = __shfl_xor_sync(0xFFFFFFFFu, best, o);
        best = v > best ? v : best;
    }
    if (lane == 0) sh.warp_mass[warp] = best;
    __syncthreads();
    if (tid < ranks) {
        for (int w = 0; w < kSampleWarps; ++w) best = sh.warp_mass[w] > best ? sh.warp_mass[w] : best;
        cluster.map_shared_rank(&sh, tid)->best[rank] = best;
    }
    cluster.sync();
    best = 0;
    for (int r = 0; r < ranks; ++r) best = sh.best[r] > best ? sh.best[r] : best;
    s.top = value_of(static_cast<uint32_t>(best >> 32));
    const uint32_t top_index = 0xFFFFFFFFu - static_cast<uint32_t>(best);
    s.temperature = p.temperature[row];
    const int top_k = p.top_k[row];
    const float top_p = p.top_p[row], min_p = p.min_p[row];

    const bool none = s.top == -INFINITY;
    if (none || !(s.temperature > 0.0f) || top_k == 1 || top_p <= 0.0f) {
        if (rank == 0 && tid == 0) {
            p.tokens[row] = none ? -1 : static_cast<int32_t>(top_index);
            if (p.probs != nullptr) p.probs[row] = none ? 0.0f : 1.0f;
        }
        return;
    }

    s.thr = Threshold{0u, 0xFFFFFFFFu};
    if (top_k > 0 && top_k < p.vocab) s.select(false, static_cast<u64>(top_k), 1.0f);
    if (top_p < 1.0f) s.select(true, 0, top_p);

    // the draw: kept masses in the order of the indices
    auto kept = [&](int i) -> u64 {
        const float l = s.logit(i);
        const uint32_t idx = s.index(i);
        if (!s.under(key_of(l), idx)) return 0;
        const float w = s.weight(l, s.depth(l));
        return w < min_p && idx != top_index ? 0 : s.mass(w);
    };
    const int seg = ((s.hi - s.lo + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32;
    const int s0 = s.lo + warp * seg, s1 = s0 + seg < s.hi ? s0 + seg : s.hi;
    u64 own = 0;
    for (int i = s0 + lane; i < s1; i += 32) own += kept(i);
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
    u64 total = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r < rank) before += sh.sum[r];
        total += sh.sum[r];
    }
    const double want = static_cast<double>(p.u[row]) * static_cast<double>(total);
    u64 target = want > 0.0 ? static_cast<u64>(want) : 0ull;
    if (target >= total) target = total - 1;
    if (target < before || target >= before + own) return;
    for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const u64 m = i < s1 ? kept(i) : 0;
        const u64 upto = before + warp_scan(m, lane);
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > target);
        if (past != 0) {
            if (lane == __ffs(past) - 1) {
                p.tokens[row] = static_cast<int32_t>(s.index(i));
                if (p.probs != nullptr) p.probs[row] = __fdiv_rn(static_cast<float>(m), static_cast<float>(total));
            }
            return;
        }
        before = __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
}

// A CTA's share of a row in shared memory: at most this many bytes.
constexpr int kSampleSmem = 16 * ((QMM_SAMPLE_MAX_VOCAB * 4 / 16 + 1 + kMaxCluster - 1) / kMaxCluster);

template <class T>
int launch(const SampleParams& p, int M, cudaStream_t stream) {
    static std::atomic<u64> configured{0};   // one bit for each device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QMM_ERR_CUDA;
    if (dev >= 64 || !(configured.load(std::memory_order_relaxed) >> dev & 1)) {
        if (cudaFuncSetAttribute(qmm_sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSampleSmem) != cudaSuccess)
            return QMM_ERR_CUDA;
        if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    int ranks = kMaxCluster;
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
    cfg.dynamicSmemBytes = static_cast<size_t>((chunks + ranks - 1) / ranks) * 16;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, qmm_sample_kernel<T>, p) == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
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
    return in_dtype == QMM_IN_F32 ? launch<float>(sp, M, st) : launch<uint16_t>(sp, M, st);
}
