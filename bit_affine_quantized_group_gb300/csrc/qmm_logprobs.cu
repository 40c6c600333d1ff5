// Log probabilities of given tokens, entropy and the largest alternatives, in
// one pass over the logits:
//   m' = max(m, l),  d = m - m',  t = (t + s d) e^d + sum e^(l - m') (l - m'),  s = s e^d + sum e^(l - m'),
//   lse = m + log s,   entropy = log s - t / s   (every term of -t is positive, so that nothing cancels).
//
// A thread keeps m, s, t and the chunk that its largest logit came from. The
// `top` best (logit, index) of a CTA's share are no worse than the `top` best of
// the threads' largest logits, and so lie with those `top` threads: their chunks
// alone, a sixteenth of the share, are read again. Each CTA of a row ranks what it
// finds by counting, the first one of the cluster ranks the CTAs' lists.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>
#include <cfloat>

#include "../../include/qmm.h"
#include "qmm_device.cuh"

namespace qmmk {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTop = QMM_LOGPROBS_MAX_TOP;
constexpr int kList = 1024;            // candidates that are ranked by counting
constexpr int kRanks = 16;             // CTAs of a row at most
constexpr int kAhead = 4;              // chunks that a thread loads before it works on the last
constexpr float kLeast = -1000.0f;     // differences are brought to it: e^-1000 is 0, and no infinity meets a 0
constexpr float kLog2E = 1.4426950408889634f;

typedef unsigned long long u64;

struct LogprobsParams {
    const void* logits;
    int64_t stride;
    const int32_t* tokens;
    float* token_logprobs;
    float* entropy;
    int32_t* top_tokens;
    float* top_logprobs;
    int32_t vocab, top;
};

struct Shared {
    u64 best[kTop];                    // of this CTA, by rank; 0 for none
    float max, sum, weighted;          // m, s and t of this CTA
    u64 all[kRanks * kTop];            // the first CTA's copy of all lists
    float stats[kRanks][3];
    u64 list[kList];
    float warp_max[kWarps], warp_sum[kWarps], warp_weighted[kWarps];
    u64 warp_best[kWarps];
    uint32_t selected[kThreads];
    uint32_t selected_size, list_size;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// NaN is -infinity, +infinity the largest float32, and -0 is 0.
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX) + 0.0f; }
// Unsigned numbers in the order of the floats, above 0.
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
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<uint16_t>(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// A row as 16-byte chunks at aligned addresses: the first and the last may hold elements outside it.
template <class T>
struct Row {
    static constexpr int kVec = 16 / sizeof(T);
    const T* base;        // of the row
    int vocab, head;      // head: elements of chunk 0 before the row
    int chunks;

    __device__ __forceinline__ Row(const T* row, int n) : base(row), vocab(n) {
        head = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        chunks = (head + n + kVec - 1) / kVec;
    }
    __device__ __forceinline__ int first(int c) const { return c * kVec - head; }
    __device__ __forceinline__ bool whole(int c) const { return first(c) >= 0 && first(c) + kVec <= vocab; }
    // chunk c, elements outside the row as -infinity
    __device__ __forceinline__ uint4 load(int c) const {
        const int e = first(c);
        if (whole(c)) return __ldg(reinterpret_cast<const uint4*>(base + e));
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const bool in = e + i >= 0 && e + i < vocab;
            if constexpr (sizeof(T) == 4) {
                w[i] = in ? __float_as_uint(base[e + i]) : 0xFF800000u;
            } else {
                const uint32_t h = in ? base[e + i] : 0xFF80u;
                w[i / 2] |= h << (16 * (i & 1));
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void values(const uint4& w, float (&v)[kVec]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = clean(__uint_as_float(u[i]));
            } else {
                v[2 * i] = clean(__uint_as_float(u[i] << 16));
                v[2 * i + 1] = clean(__uint_as_float(u[i] & 0xFFFF0000u));
            }
        }
    }
};

__device__ __forceinline__ u64 warp_max64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = w > v ? w : v;
    }
    return v;
}

template <class T>
__global__ void __launch_bounds__(kThreads, 2) qmm_logprobs_kernel(const __grid_constant__ LogprobsParams p, int ranks) {
    using R = Row<T>;
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / ranks;
    const int rank = static_cast<int>(blockIdx.x - row * ranks);
    griddep_launch_dependents();
    griddep_wait();
    const R r(static_cast<const T*>(p.logits) + row * p.stride, p.vocab);
    const int per = (r.chunks + ranks - 1) / ranks;
    const int c0 = rank * per, c1 = min(r.chunks, c0 + per);

    // the pass over the share
    float m = -INFINITY, sum = 0.0f, weighted = 0.0f;
    int at = -1;   // the chunk that m came from first
    auto take = [&](int c, const uint4& w) {
        float v[R::kVec];
        R::values(w, v);
        float most = v[0];
#pragma unroll
        for (int i = 1; i < R::kVec; ++i) most = fmaxf(most, v[i]);
        if (at < 0 || most > m) at = c;
        const float now = fmaxf(m, most), d = fmaxf(m - now, kLeast), shrink = exp2_approx(d * kLog2E);
        m = now;
        weighted = fmaf(sum, d, weighted) * shrink;
        sum *= shrink;
#pragma unroll
        for (int i = 0; i < R::kVec; ++i) {
            const float below = fmaxf(v[i] - now, kLeast), e = exp2_approx(below * kLog2E);
            sum += e;
            weighted = fmaf(e, below, weighted);
        }
    };
    uint4 next[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (c0 + tid + k * kThreads < c1) next[k] = r.load(c0 + tid + k * kThreads);
#pragma unroll 1
    for (int c = c0 + tid; c < c1; c += kAhead * kThreads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int mine = c + k * kThreads, later = mine + kAhead * kThreads;
            if (mine >= c1) break;
            const uint4 w = next[k];
            if (later < c1) next[k] = r.load(later);
            take(mine, w);
        }
    }

    // of the CTA
    float most = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    if (lane == 0) s.warp_max[warp] = most;
    if (tid == 0) s.selected_size = s.list_size = 0;
    if (tid < kTop) s.best[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) most = fmaxf(most, s.warp_max[i]);
    {
        const float d = fmaxf(m - most, kLeast), shrink = exp2_approx(d * kLog2E);
        float b = fmaf(sum, d, weighted) * shrink, a = sum * shrink;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if (lane == 0) s.warp_sum[warp] = a, s.warp_weighted[warp] = b;
    }

    if (p.top > 0) {
        // the p.top best of the threads' largest logits: the last of them is (bound, last)
        const bool some = at >= 0;
        const uint32_t key = some ? key_of(m) : 0u;
        uint32_t bound = 0;
        int last = 0x7FFFFFFF;
        if (__syncthreads_count(some) > p.top) {
            int above = 0;   // threads with key >= bound
#pragma unroll 1
            for (uint32_t bit = 0x80000000u; bit != 0; bit >>= 1) {
                const int n = __syncthreads_count(key >= (bound | bit));
                if (n >= p.top) bound |= bit, above = n;
            }
            if (above > p.top) {   // equal logits: those of the first chunks
                int low = -1;      // too few up to here
                last = r.chunks - 1;
#pragma unroll 1
                while (last - low > 1) {
                    const int mid = low + (last - low) / 2;
                    if (__syncthreads_count(key > bound || (key == bound && at <= mid)) >= p.top) last = mid;
                    else low = mid;
                }
            }
        }
        if (some && (key > bound || (key == bound && at <= last))) s.selected[atomicAdd(&s.selected_size, 1u)] = tid;
        __syncthreads();
        const int selected = static_cast<int>(s.selected_size);
        // every element of those threads that is no worse
        auto each = [&](auto&& f) {
            for (int i = warp; i < selected; i += kWarps)
                for (int c = c0 + static_cast<int>(s.selected[i]) + lane * kThreads; c < c1; c += 32 * kThreads) {
                    float v[R::kVec];
                    R::values(r.load(c), v);
#pragma unroll
                    for (int k = 0; k < R::kVec; ++k) {
                        const uint32_t q = key_of(v[k]);
                        const int e = r.first(c) + k;
                        if ((q > bound || (q == bound && c <= last)) && e >= 0 && e < p.vocab) f(entry_of(q, e));
                    }
                }
        };
        each([&](u64 entry) {
            const uint32_t slot = atomicAdd(&s.list_size, 1u);
            if (slot < kList) s.list[slot] = entry;
        });
        __syncthreads();
        const int found = static_cast<int>(s.list_size);
        if (found <= kList) {
            for (int i = tid; i < found; i += kThreads) {
                const u64 mine = s.list[i];
                int before = 0;
                for (int j = 0; j < found; ++j) before += s.list[j] > mine;
                if (before < p.top) s.best[before] = mine;
            }
        } else {   // rising logits, and the like: one after the other
            u64 previous = ~0ull;
#pragma unroll 1
            for (int k = 0; k < p.top; ++k) {
                u64 best = 0;
                each([&](u64 entry) { best = entry < previous && entry > best ? entry : best; });
                best = warp_max64(best);
                if (lane == 0) s.warp_best[warp] = best;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kWarps; ++i) best = s.warp_best[i] > best ? s.warp_best[i] : best;
                if (tid == 0) s.best[k] = best;
                previous = best;
                __syncthreads();
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) a += s.warp_sum[i], b += s.warp_weighted[i];
        s.max = most, s.sum = a, s.weighted = b;
    }

    // of the row, by its first CTA
    const u64* best = s.best;
    float total, total_weighted;
    if (ranks > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (rank == 0) {
            if (tid < ranks * kTop) s.all[tid] = cluster.map_shared_rank(s.best, tid / kTop)[tid % kTop];
            if (tid < ranks) {
                const Shared* of = cluster.map_shared_rank(&s, tid);
                s.stats[tid][0] = of->max, s.stats[tid][1] = of->sum, s.stats[tid][2] = of->weighted;
            }
        }
        cluster.sync();   // the other CTAs' memory has been read
        if (rank != 0) return;
        for (int i = 0; i < ranks; ++i) most = fmaxf(most, s.stats[i][0]);
        total = total_weighted = 0.0f;
        for (int i = 0; i < ranks; ++i) {
            const float d = fmaxf(s.stats[i][0] - most, kLeast), shrink = exp2_approx(d * kLog2E);
            total = fmaf(s.stats[i][1], shrink, total);
            total_weighted = fmaf(fmaf(s.stats[i][1], d, s.stats[i][2]), shrink, total_weighted);
        }
        if (tid < ranks * kTop) {
            const u64 mine = s.all[tid];
            int before = 0;
            for (int i = 0; i < ranks; ++i)
                for (int j = 0; j < p.top; ++j) before += s.all[i * kTop + j] > mine;
            if (mine != 0 && before < p.top) s.list[before] = mine;
        }
        // (this CTA's own list of candidates is no longer in use)
        __syncthreads();
        best = s.list;
    } else {
        __syncthreads();
        total = s.sum, total_weighted = s.weighted;
    }
    const float log_total = logf(total);
    if (tid == 0) {
        if (p.token_logprobs != nullptr) {
            const int token = p.tokens[row];
            float l = -INFINITY;
            if (token >= 0 && token < p.vocab) l = clean(to_float<T>(r.base[token]));
            p.token_logprobs[row] = l == -INFINITY ? l : (l - most) - log_total;
        }
        if (p.entropy != nullptr) p.entropy[row] = total > 0.0f ? log_total - total_weighted / total : 0.0f;
    }
    if (tid < p.top) {
        const bool in = tid < p.vocab;
        const float l = in ? value_of(static_cast<uint32_t>(best[tid] >> 32)) : -INFINITY;
        p.top_tokens[row * p.top + tid] = in ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best[tid])) : -1;
        p.top_logprobs[row * p.top + tid] = l == -INFINITY ? l : (l - most) - log_total;
    }
}

template <class T>
int launch_rows(const LogprobsParams& p, int M, cudaStream_t stream) {
    // as many CTAs for a row as fill the GPU, of 2048 logits at least
    int ranks = kRanks;
    while (ranks > 1 && (static_cast<int64_t>(M) * ranks > 2 * 152 || p.vocab / ranks < 2048)) ranks /= 2;
    if (ranks > 8) {
        static std::atomic<u64> configured{0};   // one bit for each device
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return QMM_ERR_CUDA;
        if (dev >= 64 || !(configured.load(std::memory_order_relaxed) >> dev & 1)) {
            const void* kernel = reinterpret_cast<const void*>(&qmm_logprobs_kernel<T>);
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
                return QMM_ERR_CUDA;
            if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_relaxed);
        }
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(M) * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, qmm_logprobs_kernel<T>, p, ranks) == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

}  // namespace qmmk

extern "C" int qmm_logprobs(const void* logits, int M, int vocab, int64_t stride, int in_dtype, const int32_t* tokens,
                            float* token_logprobs, float* entropy, int top, int32_t* top_tokens, float* top_logprobs,
                            void* stream) {
    using namespace qmmk;
    if (in_dtype != QMM_IN_F32 && in_dtype != QMM_IN_BF16) return QMM_ERR_INVALID_ARG;
    if (M < 0 || M > (1 << 24) || vocab < 1 || top < 0) return QMM_ERR_INVALID_ARG;
    if (vocab > QMM_SAMPLE_MAX_VOCAB || top > QMM_LOGPROBS_MAX_TOP) return QMM_ERR_UNSUPPORTED;
    if (M == 0) return QMM_OK;
    if (M > 1 && (stride < vocab || stride > (1LL << 40))) return QMM_ERR_INVALID_ARG;
    if (logits == nullptr || !aligned(logits, in_dtype == QMM_IN_F32 ? 4 : 2)) return QMM_ERR_INVALID_ARG;
    if ((tokens == nullptr) != (token_logprobs == nullptr)) return QMM_ERR_INVALID_ARG;
    if ((top > 0) != (top_tokens != nullptr) || (top > 0) != (top_logprobs != nullptr)) return QMM_ERR_INVALID_ARG;
    const void* arrays[5] = {tokens, token_logprobs, entropy, top_tokens, top_logprobs};
    for (const void* a : arrays)
        if (!aligned(a, 4)) return QMM_ERR_INVALID_ARG;
    LogprobsParams lp;
    lp.logits = logits;
    lp.stride = stride;
    lp.tokens = tokens;
    lp.token_logprobs = token_logprobs;
    lp.entropy = entropy;
    lp.top_tokens = top_tokens;
    lp.top_logprobs = top_logprobs;
    lp.vocab = vocab;
    lp.top = top;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return in_dtype == QMM_IN_F32 ? launch_rows<float>(lp, M, st) : launch_rows<uint16_t>(lp, M, st);
}
