// Log probabilities of given tokens, entropy and the largest alternatives, in
// one pass over the logits:
//   m' = max(m, l),  d = m - m',  t = (t + s d) e^d + sum e^(l - m') (l - m'),  s = s e^d + sum e^(l - m'),
//   lse = m + log s,   entropy = log s - t / s.
// For m stands a logit of the row that the largest lies less than 6 above, so that m changes seldom. Terms of -t then cancel only
// where that logit has e^-6 of the probability, and the entropy 0.017, or more; what is lost is 2^-21. (With 16 in its place
// entropies of 2e-6 were off by a fifth, and those of 512 rows by 3.9e-7 of their norm, 7.7e-8 now; 1 row took 7.3 us, with 4 7.6
// and 512 rows 25.9.) Where nothing cancels the rounding of s, 2^-24, remains.
//
// A thread keeps m, s, t, the chunk of 16 bytes that its largest logit came from
// and the largest logit of its other chunks. The `top` best (logit, index) of a
// CTA's share are no worse than the `top` best of the threads' largest logits, and
// so lie with those threads: that one chunk of theirs is read again, and all of
// them where a second one reaches as far. Each CTA of a row ranks what it finds by
// counting, the first one of the cluster ranks the CTAs' lists.
//
// One row of 151,936 float32 logits with 5 alternatives: 7.5 us, latency of the
// launch (2.2), of 10 chunks a thread, of bound, list and cluster. 512 rows of
// 100,277 bfloat16 logits with 20: 25.4 us, 4.0 TB/s, and 4 of them a row's steps
// behind the pass (21.6 without alternatives). Rows are whole: some SMs have four
// of the 512, the mean is 3.4, and four rows' instructions are about 16 us of an SM.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>
#include <cfloat>

#include "../../include/qmm.h"
#include "qmm_device.cuh"

namespace qmmk {

namespace {

namespace cg = cooperative_groups;

constexpr int kTop = QMM_LOGPROBS_MAX_TOP;
constexpr int kList = 1024;            // candidates that are ranked by counting
constexpr int kRanks = 8;              // CTAs of a row at most
// Chunks that a thread has on their way. (512 rows: four in registers 3.4 TB/s; eight here, with as many CTAs on an SM, 27.1 us, and
// twelve 32.8.)
constexpr int kAhead = 5;
constexpr int kSome = 8;               // threads that may be looked at beyond the needed ones
constexpr float kRise = 6.0f;          // that logits may lie above a thread's reference before its sums are brought to a new one
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

template <int THREADS>
struct Shared {
    u64 best[kTop];                    // of this CTA, by rank; 0 for none
    u64 all[kRanks * kTop];            // in the first CTA: the lists of all of them
    float stats[kRanks][4];            // and their m, s and t
    u64 list[kList];
    float warp_max[THREADS / 32], warp_sum[THREADS / 32], warp_weighted[THREADS / 32];
    u64 warp_best[THREADS / 32];
    uint32_t keys[THREADS];            // of the threads' largest logits; 0 for none
    int at[THREADS];                   // their chunks
    uint32_t again[THREADS];           // threads with more than that chunk to look at
    uint32_t again_size, list_size, bound;
    int last;
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
        if (whole(c)) return *reinterpret_cast<const uint4*>(base + e);
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
                v[i] = __uint_as_float(u[i]);
            } else {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            }
        }
    }
    // the largest element; NaN only where all are
    static __device__ __forceinline__ float largest(const uint4& w) {
        if constexpr (sizeof(T) == 4) {
            return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
        } else {
            auto pair = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
            const __nv_bfloat162 m = __hmax2(__hmax2(pair(w.x), pair(w.y)), __hmax2(pair(w.z), pair(w.w)));
            const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
            return fmaxf(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
        }
    }
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until no more than the last N groups of this thread are on their way
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The cluster's barrier in halves: what a thread did before its arrival is seen behind the others' waits.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

__device__ __forceinline__ u64 warp_max64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = w > v ? w : v;
    }
    return v;
}

template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) qmm_logprobs_kernel(const __grid_constant__ LogprobsParams p, int ranks) {
    using R = Row<T>;
    constexpr int kThreads = THREADS, kWarps = THREADS / 32;
    __shared__ __align__(16) Shared<THREADS> s;
    extern __shared__ __align__(16) uint4 s_ring[];   // [kAhead][thread]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / ranks;
    const int rank = static_cast<int>(blockIdx.x - row * ranks);
    if (ranks > 1) cluster_arrive();   // this CTA has started, and its memory may be written
    griddep_launch_dependents();
    griddep_wait();
    const R r(static_cast<const T*>(p.logits) + row * p.stride, p.vocab);
    const int per = (r.chunks + ranks - 1) / ranks;
    const int c0 = rank * per, c1 = min(r.chunks, c0 + per);

    // The pass over the share. Sums are held to a reference that few chunks change: the first one's largest logit, until one
    // lies kRise above it.
    float m = -INFINITY, ref = -INFINITY;
    float sums[2] = {}, weights[2] = {};   // s and t, of the even and the odd elements
    int at = -1;   // the chunk that m came from first
    float other = -INFINITY;   // the largest logit of the other chunks
    auto take = [&](int c, const uint4& w) {
        float v[R::kVec];
        R::values(w, v);
        float most = R::largest(w);   // (NaN for nothing but NaN, which changes nothing below)
        if (most > ref + kRise) {     // (also where ref is still -infinity, and for an infinity, which becomes the largest number)
            if (most == INFINITY) {
                most = FLT_MAX;
#pragma unroll
                for (int i = 0; i < R::kVec; ++i) v[i] = clean(v[i]);
            }
            const float d = fmaxf(ref - most, kLeast), shrink = exp2_approx(d * kLog2E);
            ref = most;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                weights[i] = fmaf(sums[i], d, weights[i]) * shrink;
                sums[i] *= shrink;
            }
        }
        if (most > m) at = c;
        other = fmaxf(other, fminf(m, most));
        m = fmaxf(m, most);
        const float less = -ref;
#pragma unroll
        for (int i = 0; i < R::kVec; i += 2) {   // (NaN - ref and -infinity - -infinity come to kLeast too)
            float x[2], e[2];
            add_x2(x[0], x[1], v[i], v[i + 1], less, less);
            x[0] = fmaxf(x[0], kLeast), x[1] = fmaxf(x[1], kLeast);
            mul_x2(e[0], e[1], x[0], x[1], kLog2E, kLog2E);
            e[0] = exp2_approx(e[0]), e[1] = exp2_approx(e[1]);
            add_x2(sums[0], sums[1], sums[0], sums[1], e[0], e[1]);
            fma_x2(weights[0], weights[1], e[0], e[1], x[0], x[1], weights[0], weights[1]);
        }
    };
    // the row's first and last chunk may be cut short
    const int w0 = max(c0, r.whole(0) ? 0 : 1), w1 = min(c1, r.whole(r.chunks - 1) ? r.chunks : r.chunks - 1);
    const uint4* const chunks = reinterpret_cast<const uint4*>(r.base - r.head);
    // every thread reads what it has copied itself, and refills a place when what it held has been used
    const uint32_t ring = smem_u32(s_ring + tid);
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k) {
        const int c = w0 + tid + k * kThreads;
        if (c < w1) cp_async_16(ring + k * (kThreads * 16), chunks + c);
        cp_async_commit();
    }
    const bool with_first = tid == 0 && c0 < w0 && c0 < c1, with_last = tid == 1 && w1 < c1 && w1 >= w0;
    // (the first of its chunks, where none has a logit above -infinity)
    at = with_first ? c0 : w0 + tid < w1 ? w0 + tid : with_last ? w1 : -1;
    if (with_first) take(c0, r.load(c0));
    const uint4* ahead = chunks + w0 + tid + (kAhead - 1) * kThreads;
#pragma unroll 1
    for (int c = w0 + tid; c < w1; c += kAhead * kThreads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int mine = c + k * kThreads;
            if (mine >= w1) break;
            if (mine + (kAhead - 1) * kThreads < w1) cp_async_16(ring + (k + kAhead - 1) % kAhead * (kThreads * 16), ahead);
            cp_async_commit();
            ahead += kThreads;
            cp_async_wait<kAhead - 1>();
            take(mine, s_ring[k * kThreads + tid]);
        }
    }
    if (with_last) take(w1, r.load(w1));   // (after the others: `at` is the first of equal ones)
    m += 0.0f;
    const float sum = sums[0] + sums[1], weighted = weights[0] + weights[1];

    // of the CTA
    float most = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    if (lane == 0) s.warp_max[warp] = most;
    if (tid == 0) s.again_size = s.list_size = 0;
    const uint32_t key = at >= 0 ? key_of(m) : 0u;
    s.keys[tid] = key;
    s.at[tid] = at;
    if (tid < kTop) s.best[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) most = fmaxf(most, s.warp_max[i]);
    {
        const float d = fmaxf(ref - most, kLeast), shrink = exp2_approx(d * kLog2E);
        float b = fmaf(sum, d, weighted) * shrink, a = sum * shrink;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if (lane == 0) s.warp_sum[warp] = a, s.warp_weighted[warp] = b;
    }

    if (p.top > 0) {
        // a bound that the largest logits of p.top threads reach, and of few more: (bound, last). By one warp, for it costs the
        // same time and less of the other rows'.
        if (warp == 0) {
            // (the largest of every few threads do: p.top of them are p.top threads)
            constexpr int kKeys = 4, kOf = kWarps / kKeys;
            uint32_t keys[kKeys], low_key = 0xFFFFFFFFu, high_key = 0;
            int count = 0;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                keys[i] = 0;
#pragma unroll
                for (int j = 0; j < kOf; ++j) keys[i] = max(keys[i], s.keys[(i * kOf + j) * 32 + lane]);
                if (keys[i] != 0) low_key = min(low_key, keys[i]);
                high_key = max(high_key, keys[i]);
                count += keys[i] != 0;
            }
            low_key = __reduce_min_sync(0xFFFFFFFFu, low_key);
            high_key = __reduce_max_sync(0xFFFFFFFFu, high_key);
            int reach = __reduce_add_sync(0xFFFFFFFFu, count);   // of them with key >= bound
            uint32_t bound = 0;
            int last = 0x7FFFFFFF;
            if (reach > p.top + kSome) {
                // bit by bit below the first that the keys differ in
                const uint32_t differ = low_key ^ high_key;
                bound = low_key & ~(differ == 0 ? 0u : 0xFFFFFFFFu >> __clz(differ));
#pragma unroll 1
                for (uint32_t bit = differ == 0 ? 0u : 0x80000000u >> __clz(differ); bit != 0 && reach > p.top + kSome; bit >>= 1) {
                    int n = 0;
#pragma unroll
                    for (int i = 0; i < kKeys; ++i) n += keys[i] >= (bound | bit);
                    n = __reduce_add_sync(0xFFFFFFFFu, n);
                    if (n >= p.top) bound |= bit, reach = n;
                }
                if (reach > p.top + kSome) {   // equal logits: those of the first chunks
                    int low = -1;              // too few up to here
                    last = r.chunks - 1;
#pragma unroll 1
                    while (last - low > 1) {
                        const int mid = low + (last - low) / 2;
                        int n = 0;
#pragma unroll 1
                        for (int i = 0; i < kWarps; ++i)
                            n += s.keys[i * 32 + lane] > bound || (s.keys[i * 32 + lane] == bound && s.at[i * 32 + lane] <= mid);
                        n = __reduce_add_sync(0xFFFFFFFFu, n);
                        if (n >= p.top) last = mid;
                        else low = mid;
                    }
                }
            }
            if (lane == 0) s.bound = bound, s.last = last;
        }
        __syncthreads();
        const uint32_t bound = s.bound;
        const int last = s.last;
        const float bound_value = bound <= key_of(-INFINITY) ? -INFINITY : value_of(bound);
        // every element of a chunk that is no worse
        auto look = [&](int c, const uint4& w, auto&& f) {
            if (!(fmaxf(R::largest(w), -INFINITY) >= bound_value)) return;
            float v[R::kVec];
            R::values(w, v);
#pragma unroll
            for (int k = 0; k < R::kVec; ++k) {
                const uint32_t q = key_of(clean(v[k]));
                const int e = r.first(c) + k;
                if ((q > bound || (q == bound && c <= last)) && e >= 0 && e < p.vocab) f(entry_of(q, e));
            }
        };
        // the chunks of the threads `again`, and with `all` those of their largest logits too
        auto each = [&](bool all, auto&& f) {
            const int count = static_cast<int>(s.again_size);
            for (int i = warp; i < count; i += kWarps) {
                const int of = static_cast<int>(s.again[i]), seen = all ? -1 : s.at[of];
                for (int c = w0 + of + lane * kThreads; c < w1; c += 32 * kThreads)
                    if (c != seen) look(c, chunks[c], f);
                if (lane == 0 && of == 0 && c0 < w0 && c0 < c1 && c0 != seen) look(c0, r.load(c0), f);
                if (lane == 0 && of == 1 && w1 < c1 && w1 >= w0 && w1 != seen) look(w1, r.load(w1), f);
            }
        };
        auto note = [&](u64 entry) {
            const uint32_t slot = atomicAdd(&s.list_size, 1u);
            if (slot < kList) s.list[slot] = entry;
        };
        const bool mine = key > bound || (key == bound && at <= last && at >= 0);
        // (the threads' own chunks are on their way while it is settled which others are to be looked at)
        uint4 own = make_uint4(0u, 0u, 0u, 0u);
        if (mine) {
            // (of short shares it is still where it was copied to)
            const bool held = w1 - w0 <= kAhead * kThreads && at >= w0 && at < w1;
            own = held ? s_ring[at - w0] : r.load(at);
            if (other >= bound_value) s.again[atomicAdd(&s.again_size, 1u)] = tid;
        }
        __syncthreads();
        if (s.again_size != 0) each(false, note);
        if (mine) look(at, own, note);
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
            __syncthreads();   // every thread has seen how many are to be looked at again
            if (mine && !(other >= bound_value)) s.again[atomicAdd(&s.again_size, 1u)] = tid;
            __syncthreads();
            u64 previous = ~0ull;
#pragma unroll 1
            for (int k = 0; k < p.top; ++k) {
                u64 best = 0;
                each(true, [&](u64 entry) { best = entry < previous && entry > best ? entry : best; });
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
    float total = 0.0f, total_weighted = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total += s.warp_sum[i], total_weighted += s.warp_weighted[i];

    // of the row, by its first CTA
    const u64* best = s.best;
    if (ranks > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster_wait();   // the first CTA has started
        if (tid < kTop) *cluster.map_shared_rank(&s.all[rank * kTop + tid], 0) = s.best[tid];
        if (tid == 0) *cluster.map_shared_rank(reinterpret_cast<float4*>(s.stats[rank]), 0) = make_float4(most, total, total_weighted, 0.0f);
        cluster_arrive();
        if (rank != 0) return;
        cluster_wait();
        for (int i = 0; i < ranks; ++i) most = fmaxf(most, s.stats[i][0]);
        total = total_weighted = 0.0f;
        for (int i = 0; i < ranks; ++i) {
            const float d = fmaxf(s.stats[i][0] - most, kLeast), shrink = exp2_approx(d * kLog2E);
            total = fmaf(s.stats[i][1], shrink, total);
            total_weighted = fmaf(fmaf(s.stats[i][1], d, s.stats[i][2]), shrink, total_weighted);
        }
        // (this CTA's own list of candidates is no longer in use)
        for (int j = tid; j < ranks * kTop; j += kThreads) {
            const u64 mine = s.all[j];
            if (mine == 0) continue;
            int before = 0;
            for (int i = 0; i < ranks; ++i)
                for (int k = 0; k < p.top; ++k) before += s.all[i * kTop + k] > mine;
            if (before < p.top) s.list[before] = mine;
        }
        __syncthreads();
        best = s.list;
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

template <class T, int THREADS>
int launch(const LogprobsParams& p, int M, int ranks, cudaStream_t stream) {
    static std::atomic<u64> configured{0};   // one bit for each device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QMM_ERR_CUDA;
    if (dev >= 64 || !(configured.load(std::memory_order_relaxed) >> dev & 1)) {
        const void* kernel = reinterpret_cast<const void*>(&qmm_logprobs_kernel<T, THREADS>);
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, THREADS * kAhead * 16) != cudaSuccess)
            return QMM_ERR_CUDA;
        if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(M) * ranks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = THREADS * kAhead * 16;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, qmm_logprobs_kernel<T, THREADS>, p, ranks) == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

template <class T>
int launch_rows(const LogprobsParams& p, int M, cudaStream_t stream) {
    // CTAs of 512 threads while two an SM hold all rows, as clusters of them where that leaves each 16,384 logits and not much
    // more than seven eighths of the places taken: of clusters that fill the GPU some wait. (151,936 bfloat16 logits, 20
    // alternatives, 1, 2, 4 and 8 CTAs a row: 1 row 11.4, 9.4, 8.3 and 8.3 us, 8 rows 9.8, 8.6 and 9.3 for the last three, 64
    // rows 15.6, 13.9 and 11.7, 76 rows 12.3, 10.3 and 16.8; 16 CTAs a row 11.1 for one. 32,000 logits: 5.5 to 6 us as one.)
    // More rows: CTAs of 256, so that one's steps behind the pass and the last rows' overhang cost little. (256 rows: 20.3 us,
    // as two CTAs of 256 each 23.6, as one 31. 400 of 100,277: 24.1 as one CTA of 256 each.)
    constexpr int kCtas = 2 * 152;
    if (M > kCtas) return launch<T, 256>(p, M, 1, stream);
    int ranks = M <= 6 ? kRanks : kRanks / 2;
    while (ranks > 1 && (M * ranks > kCtas * 7 / 8 || p.vocab / ranks < 16384)) ranks /= 2;
    return launch<T, 512>(p, M, ranks, stream);
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
