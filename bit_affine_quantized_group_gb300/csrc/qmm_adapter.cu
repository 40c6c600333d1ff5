// Low-rank adapters of many requests beside a projection that they share:
//   low[m, :] = scale[i] * x[m, :] A[i]^T,   out[m, :] = y[m, :] + low[m, :] B[i]^T,   i = ids[m].
//
// Both products are m16n8k16 tensor-core products of up to 16 rows of one
// adapter: the rows of a block of 64 are put in the order of their adapters and
// cut into such tiles, which every CTA does for itself. Their bound is bytes: A
// and B of the adapters in use once, x, y and out; of few rows latency, so that
// every warp has all its loads on their way at once.
//   - low: the warps of a cluster's CTAs take a tile's 16 columns of rank each,
//     the CTAs slices of K. They write their sums into the shared memory of the
//     CTA that a row belongs to, which adds them in the order of the slices.
//   - out: each warp takes a run of a tile's columns, 32 at a time. low enters as
//     two bfloat16 terms (high + low within 2^-17), for float32 outputs as three
//     (2^-26): one would round more than bfloat16 outputs do. Tiles, y and B are
//     read while the first kernel still runs. That one lets the second start only
//     behind its own wait, when all that came before the call is complete; but
//     sight of it is promised behind the second's wait alone. So ids and the first
//     y are read from L2, where a completed kernel's writes are, past any older
//     line of an SM's own cache.
// In both a lane of a quad has 8 neighbouring elements of the 32 that two
// products sum over, so that loads are whole 16-byte vectors of whole sectors.
// K 4096, N 6144, a row for each of 16 adapters of rank 16: 7.0 us, of which 4.2
// are the first kernel and 2.2 a launch. 64 rows of 16 adapters of rank 64, K
// 5120, N 17408, float32: 19.1 us. 2048 rows, rank 32, K 5120, N 6144: 23.2 us
// (3.2 TB/s), 11.3 of them the first kernel: both wait for loads, of which a
// lane's registers hold no more, and which are more than the operands, for A and
// B are read again for every tile of 16 rows. (Tried there: loads of the step five on as soon
// as a step's products run, y through a ring of asynchronous copies, no gain;
// 32 columns of rank a unit, with two warps on a unit's K: 1 us more, 5 % less
// for 16,000 rows of rank 64.)
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <pthread.h>

#include <atomic>
#include <cmath>
#include <new>
#include <type_traits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"

struct qmm_adapter_plan {
    qmm_adapter_desc d;
    int device;
    int num_sms;
    uint8_t* ws;
    bool owns_ws;
    // held while a call launches: its second kernel reads what its first left in the workspace, and no other thread's call may
    // come between the two
    mutable pthread_mutex_t launches = PTHREAD_MUTEX_INITIALIZER;
};

namespace qmmk {

namespace {

namespace cg = cooperative_groups;

constexpr int kBlock = 64;            // rows whose adapters are put in order
constexpr int kTile = 16;             // rows of a product
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlices = 16;           // of K at most: the CTAs of a cluster
// Clusters of 16 CTAs that run at once; more of them wait. (64 rows of rank 64: 5.5 us with clusters of 8, 8.5 with 16 of 16;
// 16 rows of rank 16, which need two: 5.2 and 4.2.)
constexpr int kWideClusters = 8;
constexpr int kStep = 32;             // elements that two products sum over
constexpr int kAhead = 5;             // steps of K that a warp loads at once
constexpr size_t kErrBytes = 256;

constexpr int terms_of(int out_dtype) { return out_dtype == QMM_OUT_F32 ? 3 : 2; }

struct AdapterParams {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scale;
    const int32_t* ids;
    const void* y;
    void* out;
    uint16_t* low;           // [term][rows][rank] bfloat16
    int64_t low_term;        // elements from term to term
    uint32_t* err;
    int64_t x_stride, y_stride, out_stride;
    int64_t K, N;
    int32_t rank, adapters, rows;
};

// The rows of a block in the order of their adapters (-1 first), and the tiles of up to 16 of one adapter.
struct Tiles {
    int4 id[kBlock / 4];     // of the rows as they stand
    uint8_t row[kBlock];     // at each place of the order
    int32_t tile_id[kBlock];
    uint8_t first[kBlock], size[kBlock];   // places of a tile
    uint8_t tile[kBlock];    // of a place
    uint32_t starts[2];
    int tiles;
};

// By the whole CTA; ids outside -1..adapters-1 count as -1.
__device__ __forceinline__ void find_tiles(const AdapterParams& p, int row0, Tiles& t) {
    const int tid = threadIdx.x, rows = min(kBlock, p.rows - row0);
    if (tid < kBlock) {
        int id = 0x7FFFFFFF;   // behind all others
        if (tid < rows) {
            id = __ldcg(p.ids + row0 + tid);
            if (id < -1 || id >= p.adapters) {
                atomicOr(p.err, static_cast<uint32_t>(QMM_ADAPTER_BAD_ID));
                id = -1;
            }
        }
        reinterpret_cast<int32_t*>(t.id)[tid] = id;
        if (tid < 2) t.starts[tid] = 0;
        named_barrier(1, kBlock);
        int before = 0, same = 0;   // rows of smaller ids, and earlier rows of this one
#pragma unroll
        for (int j = 0; j < kBlock; j += 4) {
            const int4 other = t.id[j / 4];
            before += (other.x < id) + (other.y < id) + (other.z < id) + (other.w < id);
            same += (other.x == id && j < tid) + (other.y == id && j + 1 < tid) + (other.z == id && j + 2 < tid) +
                    (other.w == id && j + 3 < tid);
        }
        const int place = before + same;
        if (tid < rows) t.row[place] = static_cast<uint8_t>(tid);
        // which places begin a tile
        const bool begins = tid < rows && same % kTile == 0;
        if (begins) atomicOr(&t.starts[place >> 5], 1u << (place & 31));
        named_barrier(1, kBlock);
        const uint32_t s0 = t.starts[0], s1 = t.starts[1];
        const uint64_t starts = static_cast<uint64_t>(s1) << 32 | s0;
        if (begins) {
            const uint64_t below = (1ull << place) - 1, after = place == 63 ? 0 : starts >> (place + 1);
            const int tile = __popcll(starts & below);
            const int next = after == 0 ? rows : place + __ffsll(static_cast<long long>(after));
            t.tile_id[tile] = id;
            t.first[tile] = static_cast<uint8_t>(place);
            t.size[tile] = static_cast<uint8_t>(next - place);
        }
        if (tid < rows) t.tile[place] = static_cast<uint8_t>(__popcll(starts & (0xFFFFFFFFFFFFFFFFull >> (63 - place))) - 1);
        if (tid == 0) t.tiles = __popc(s0) + __popc(s1);
    }
    __syncthreads();
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// v as bfloat16 terms of falling size; an infinity or NaN stands in the first alone.
template <int TERMS>
__device__ __forceinline__ void split(float v, uint32_t (&term)[TERMS]) {
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        const float f = __bfloat162float(h);
        term[i] = __bfloat16_as_ushort(h);
        v = fabsf(f) < INFINITY ? v - f : 0.0f;
    }
}

__device__ __forceinline__ uint4 load16(const uint16_t* p, bool in) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (in) v = load_written(p);
    return v;
}
__device__ __forceinline__ uint4 load_weights(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Two products of fragments that hold 8 neighbouring elements a lane: rows a0 (gid) and a1 (gid + 8), column gid of b.
__device__ __forceinline__ void mma_32(float (&d)[4], const uint4& a0, const uint4& a1, const uint4& b) {
    const uint32_t first[4] = {a0.x, a1.x, a0.y, a1.y}, second[4] = {a0.z, a1.z, a0.w, a1.w};
    mma_bf16(d, first, b.x, b.y);
    mma_bf16(d, second, b.z, b.w);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Grid: clusters of `slices` CTAs; block of rows, then one of `groups` that share its units (a tile's 16 columns of rank).
template <int TERMS>
__global__ void __launch_bounds__(kThreads, 2) qmm_adapter_low_kernel(const __grid_constant__ AdapterParams p, int slices, int groups) {
    // The sums of the places `slice`, `slice` + slices, ... from every CTA of the cluster: [place / slices][slice][rank].
    // (slices is a power of two)
    extern __shared__ __align__(16) float s_part[];
    __shared__ __align__(16) Tiles t;
    __shared__ float s_scale[kBlock];   // of the tiles
    cg::cluster_group cluster = cg::this_cluster();
    const int slice = static_cast<int>(blockIdx.x % slices), of = static_cast<int>(blockIdx.x / slices);
    const int group = of % groups, row0 = of / groups * kBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, quad = lane & 3;
    cluster_arrive();   // this CTA has started, and its memory may be written
    griddep_wait();
    griddep_launch_dependents();   // not before: the second kernel reads what came before this one without waiting
    const uint16_t* const p_a = behind_wait(p.a);
    const uint16_t* const p_x = behind_wait(p.x);
    find_tiles(p, row0, t);
    float scale = 1.0f;   // (on its way while the products run)
    if (p.scale != nullptr && threadIdx.x < t.tiles && t.tile_id[threadIdx.x] >= 0) scale = __ldg(p.scale + t.tile_id[threadIdx.x]);
    cluster_wait();
    const int columns = (p.rank + 15) / 16, units = t.tiles * columns;
    const int steps = static_cast<int>(p.K / kStep);
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * slice / slices);
    const int count = static_cast<int>(static_cast<int64_t>(steps) * (slice + 1) / slices) - s0;

    for (int u = group + warp * groups; u < units; u += kWarps * groups) {
        const int tile = u / columns, column = (u - tile * columns) * 16, id = t.tile_id[tile];
        if (id < 0) continue;
        const int first = t.first[tile], size = t.size[tile];
        const bool two = column + 8 < p.rank;
        const uint16_t* const a = p_a + (static_cast<int64_t>(id) * p.rank + column + gid) * p.K + s0 * kStep + quad * 8;
        const int64_t a_next = 8 * p.K;
        const uint16_t* x[2];
        bool in[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            in[h] = gid + 8 * h < size;
            x[h] = p_x + static_cast<int64_t>(row0 + (in[h] ? t.row[first + gid + 8 * h] : 0)) * p.x_stride + s0 * kStep + quad * 8;
        }
        float acc[2][4] = {};
        for (int k0 = 0; k0 < count; k0 += kAhead) {
            uint4 wa[kAhead][2], wx[kAhead][2];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool some = k0 + k < count;
                const int at = (k0 + k) * kStep;
                wa[k][0] = load16(a + at, some);
                wa[k][1] = load16(a + a_next + at, some && two);
                wx[k][0] = load16(x[0] + at, some && in[0]);
                wx[k][1] = load16(x[1] + at, some && in[1]);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                mma_32(acc[0], wx[k][0], wx[k][1], wa[k][0]);
                mma_32(acc[1], wx[k][0], wx[k][1], wa[k][1]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!in[h]) continue;
            const int place = first + gid + 8 * h, owner = place & (slices - 1);
            float* const to = cluster.map_shared_rank(s_part, owner) + (place - owner + slice) * p.rank + column + quad * 2;
            *reinterpret_cast<float2*>(to) = make_float2(acc[0][2 * h], acc[0][2 * h + 1]);
            if (two) *reinterpret_cast<float2*>(to + 8) = make_float2(acc[1][2 * h], acc[1][2 * h + 1]);
        }
    }
    if (threadIdx.x < kBlock) s_scale[threadIdx.x] = scale;
    cluster_arrive();
    cluster_wait();
    // a place for each warp, two columns for each lane, of the units of this group
    const int rows = min(kBlock, p.rows - row0);
    for (int place = slice + warp * slices; place < rows; place += kWarps * slices) {
        const int tile = t.tile[place], id = t.tile_id[tile];
        if (id < 0) continue;
        const float by = s_scale[tile];
        const int64_t at = static_cast<int64_t>(row0 + t.row[place]) * p.rank;
        for (int c = 2 * lane; c < p.rank; c += 64) {
            if ((tile * columns + c / 16) % groups != group) continue;
            const float* from = s_part + (place - slice) * p.rank + c;
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 4
            for (int i = 0; i < slices; ++i, from += p.rank) {
                const float2 v = *reinterpret_cast<const float2*>(from);
                sum.x += v.x;
                sum.y += v.y;
            }
            uint32_t x[TERMS], y[TERMS];
            split(sum.x * by, x);
            split(sum.y * by, y);
#pragma unroll
            for (int i = 0; i < TERMS; ++i) *reinterpret_cast<uint32_t*>(p.low + i * p.low_term + at + c) = x[i] | y[i] << 16;
        }
    }
}

template <bool F32, int STEPS>
constexpr bool staged = F32 || STEPS == 4;
template <bool F32, int STEPS>
constexpr int low_bytes = staged<F32, STEPS> ? STEPS * (F32 ? 3 : 2) * 2 * kThreads * 16 : 0;

// A run of units of a tile's 32 columns for each warp; a lane has 8 neighbouring columns of two rows. STEPS: 32 elements of
// rank each. WIDE: rows of y and out are read and written 16 bytes at a time.
template <bool F32, int STEPS, bool WIDE>
__global__ void __launch_bounds__(kThreads, STEPS == 1 && !F32 ? 3 : 2) qmm_adapter_out_kernel(const __grid_constant__ AdapterParams p, int groups) {
    constexpr int kTerms = F32 ? 3 : 2;
    // low stays over a tile's units, in registers or in shared memory: that leaves registers for the next unit's B and y to be
    // loaded as soon as this one's have been used. (64 rows of rank 64 in float32: 18.8 us, 19.1 without; 2048 of rank 128: 79
    // and 113. 2048 rows of rank 32 in bfloat16, whose terms are fewer: 24.0 and 22.8.)
    constexpr bool kStage = staged<F32, STEPS>;
    extern __shared__ __align__(16) uint4 s_low[];   // [warp][step][term][row][lane]
    __shared__ __align__(16) Tiles t;
    using T = std::conditional_t<F32, float, uint16_t>;
    const int group = static_cast<int>(blockIdx.x % groups), row0 = static_cast<int>(blockIdx.x / groups) * kBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, quad = lane & 3;
    griddep_launch_dependents();
    find_tiles(p, row0, t);   // (before the wait, as the first y and B: what is read there was complete when the first kernel began)
    const uint32_t columns = static_cast<uint32_t>((p.N + 31) / 32);
    const uint32_t units = t.tiles * columns;   // (2^31 at most)
    const uint32_t all = groups * kWarps, mine = group * kWarps + warp, each = units / all, rest = units - each * all;
    uint32_t u = mine * each + min(mine, rest);
    const uint32_t u1 = u + each + (mine < rest ? 1 : 0);
    bool waited = false;   // for the first kernel
    while (u < u1) {
        const int tile = static_cast<int>(u / columns);
        uint32_t column = u - tile * columns;
        const uint32_t end = min(column + (u1 - u), columns);
        u += end - column;
        const int id = t.tile_id[tile], first = t.first[tile], size = t.size[tile];
        if (id < 0 && p.y == p.out) continue;
        bool in[2];
        const T* y[2];
        T* out[2];
        const uint16_t* low[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            in[h] = gid + 8 * h < size;
            const int64_t row = row0 + (in[h] ? t.row[first + gid + 8 * h] : 0);
            // of the lane's first column of the unit
            y[h] = static_cast<const T*>(p.y) + row * p.y_stride + static_cast<int64_t>(column) * 32 + quad * 8;
            out[h] = static_cast<T*>(p.out) + row * p.out_stride + static_cast<int64_t>(column) * 32 + quad * 8;
            low[h] = p.low + row * p.rank + quad * 8;
        }
        // the columns of a unit: 8 (gid / 2) + 2 j + gid % 2 for the product j, so that a lane gets the 8 from 8 quad on
        const int own = 8 * (gid >> 1) + (gid & 1);
        const uint16_t* b = p.b + (static_cast<int64_t>(id < 0 ? 0 : id) * p.N + static_cast<int64_t>(column) * 32 + own) * p.rank + quad * 8;
        const int b_next = 2 * p.rank;
        bool in_rank[STEPS];   // this lane's elements are there
#pragma unroll
        for (int k = 0; k < STEPS; ++k) in_rank[k] = id >= 0 && k * 32 + quad * 8 < p.rank;
        const bool all_rank = id >= 0 && p.rank == 32 * STEPS;
        uint4 l[kStage ? 1 : STEPS][kTerms][2];
        bool loaded = false;
        uint4 wy[2][F32 ? 2 : 1], wb[STEPS][4];   // y and B of a unit
        auto load_y = [&](int ahead, int left, bool early) {   // early: before the wait
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < (F32 ? 2 : 1); ++k)
                    if (WIDE && in[h] && quad * 8 + 8 <= left) {
                        const uint4* const from = reinterpret_cast<const uint4*>(y[h] + ahead + 4 * k);
                        wy[h][k] = F32 && !early ? *from : __ldcg(from);   // (of float32 two loads share a sector)
                    }
        };
        auto load_b = [&](const uint16_t* from, int left) {
            if (all_rank && left == 32) {
#pragma unroll
                for (int k = 0; k < STEPS; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) wb[k][j] = load_weights(from + j * b_next + k * 32);
            } else {
#pragma unroll
                for (int k = 0; k < STEPS; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) wb[k][j] = in_rank[k] && own + 2 * j < left ? load_weights(from + j * b_next + k * 32) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        auto columns_of = [&](uint32_t c) { return static_cast<int>(min(p.N - static_cast<int64_t>(c) * 32, static_cast<int64_t>(32))); };
        int left = columns_of(column);
        if constexpr (kStage) load_y(0, left, !waited), load_b(b, left);
#pragma unroll 1
        for (; column < end; ++column, b += 16 * b_next, y[0] += 32, y[1] += 32, out[0] += 32, out[1] += 32) {
            const bool whole = WIDE && quad * 8 + 8 <= left;
            const bool more = column + 1 < end;
            const int left_next = more ? columns_of(column + 1) : 0;
            const bool roll = kStage && more && all_rank && left_next == 32;
            if constexpr (!kStage) load_y(0, left, !waited), load_b(b, left);
            if (!waited) {
                griddep_wait();
                waited = true;
            }
            if (!loaded) {
                loaded = true;
#pragma unroll
                for (int k = 0; k < STEPS; ++k)
#pragma unroll
                    for (int i = 0; i < kTerms; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint4 v = make_uint4(0u, 0u, 0u, 0u);
                            if (in[h] && in_rank[k]) v = __ldcg(reinterpret_cast<const uint4*>(low[h] + i * p.low_term + k * 32));
                            if constexpr (kStage) s_low[(((warp * STEPS + k) * kTerms + i) * 2 + h) * 32 + lane] = v;
                            else l[k][i][h] = v;
                        }
            }
            float acc[4][4] = {};
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                uint4(&lk)[kTerms][2] = l[kStage ? 0 : k];
                if constexpr (kStage) {   // (each lane what it has written itself)
#pragma unroll
                    for (int i = 0; i < kTerms; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) lk[i][h] = s_low[(((warp * STEPS + k) * kTerms + i) * 2 + h) * 32 + lane];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < kTerms; ++i) mma_32(acc[j], lk[i][0], lk[i][1], wb[k][j]);
                if (roll) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) wb[k][j] = load_weights(b + 16 * b_next + j * b_next + k * 32);
                }
            }
            if (kStage && more && !roll) load_b(b + 16 * b_next, left_next);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!in[h]) continue;
                if (whole) {
                    if constexpr (F32) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint4& v = wy[h][k];
                            *reinterpret_cast<float4*>(out[h] + 4 * k) = make_float4(
                                __uint_as_float(v.x) + acc[2 * k][2 * h], __uint_as_float(v.y) + acc[2 * k][2 * h + 1],
                                __uint_as_float(v.z) + acc[2 * k + 1][2 * h], __uint_as_float(v.w) + acc[2 * k + 1][2 * h + 1]);
                        }
                    } else {
                        const uint32_t w[4] = {wy[h][0].x, wy[h][0].y, wy[h][0].z, wy[h][0].w};
                        uint32_t r[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            r[j] = pack_bf16(__uint_as_float(w[j] << 16) + acc[j][2 * h],
                                             __uint_as_float(w[j] & 0xFFFF0000u) + acc[j][2 * h + 1]);
                        *reinterpret_cast<uint4*>(out[h]) = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (quad * 8 + j >= left) break;
                        const float add = acc[j >> 1][2 * h + (j & 1)];
                        if constexpr (F32) out[h][j] = y[h][j] + add;
                        else
                            out[h][j] = static_cast<uint16_t>(
                                pack_bf16(__uint_as_float(static_cast<uint32_t>(y[h][j]) << 16) + add, 0.0f));
                    }
                }
            }
            if (kStage && more) load_y(32, left_next, false);
            left = left_next;
        }
    }
    if (!waited) griddep_wait();   // (the next kernel must not start behind a first kernel that still runs)
}

template <int TERMS>
cudaError_t launch_low(const AdapterParams& p, int num_sms, cudaStream_t stream) {
    const int64_t blocks = (p.rows + kBlock - 1) / kBlock;
    const int64_t steps = p.K / kStep;
    // two CTAs an SM; units of a block: one for each 16 columns of rank of up to as many tiles as it has rows
    const int64_t units = static_cast<int64_t>(p.rows < kBlock ? p.rows : kBlock) * ((p.rank + 15) / 16);
    const int64_t most = (units + kWarps - 1) / kWarps;
    int slices = blocks * most <= kWideClusters ? kSlices : kSlices / 2;
    // of clusters that fill the GPU some wait: 1216 rows of one adapter of rank 32 took 22.7 us with 304 CTAs, 17.2 with 152
    const int64_t places = 2 * num_sms * 7 / 8;
    while (slices > 1 && (slices > steps || slices * blocks > places)) slices /= 2;
    int64_t groups = (slices > 1 ? places : 2 * num_sms) / (blocks * slices);
    groups = groups < 1 ? 1 : groups > most ? most : groups;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(slices);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * groups * slices));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>((kBlock + slices - 1) / slices * slices) * p.rank * 4;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, qmm_adapter_low_kernel<TERMS>, p, slices, static_cast<int>(groups));
}

template <bool F32, int STEPS, bool WIDE>
cudaError_t launch_out_steps(const AdapterParams& p, int num_sms, cudaStream_t stream) {
    const int64_t blocks = (p.rows + kBlock - 1) / kBlock;
    const int64_t units = (p.rows < kBlock ? p.rows : kBlock) * ((p.N + 31) / 32);
    // As many CTAs as run at once, or up to four times as many: what takes least where a warp's unit and a CTA's start take one
    // each. (2048 rows: 22.9 us, with 24 CTAs more than run at once 27.4; 19,456 rows, 304 blocks: 123 with three rounds of
    // CTAs, 140 with one.)
    const int64_t most = (units + kWarps - 1) / kWarps, slots = (STEPS == 1 && !F32 ? 3 : 2) * num_sms;
    const int64_t work = ((p.rows < kBlock ? 1 : kBlock / kTile) * ((p.N + 31) / 32) + kWarps - 1) / kWarps;   // of a warp, at least
    int64_t groups = 1, least = INT64_MAX;
    for (int rounds = 1; rounds <= 4; ++rounds) {
        int64_t g = rounds * slots / blocks;
        g = g < 1 ? 1 : g > most ? most : g;
        const int64_t cost = (blocks * g + slots - 1) / slots * ((work + g - 1) / g + 1);
        if (cost < least) least = cost, groups = g;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * groups));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = low_bytes<F32, STEPS>;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qmm_adapter_out_kernel<F32, STEPS, WIDE>, p, static_cast<int>(groups));
}

template <bool F32>
cudaError_t launch_out(const AdapterParams& p, bool wide, int num_sms, cudaStream_t stream) {
    auto with = [&](auto steps) -> cudaError_t {
        constexpr int STEPS = decltype(steps)::value;
        return wide ? launch_out_steps<F32, STEPS, true>(p, num_sms, stream) : launch_out_steps<F32, STEPS, false>(p, num_sms, stream);
    };
    if (p.rank <= 32) return with(std::integral_constant<int, 1>());
    if (p.rank <= 64) return with(std::integral_constant<int, 2>());
    return with(std::integral_constant<int, 4>());
}

template <bool F32, int STEPS>
cudaError_t configure_out() {
    if (low_bytes<F32, STEPS> <= 32 * 1024) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(qmm_adapter_out_kernel<F32, STEPS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, low_bytes<F32, STEPS>);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(qmm_adapter_out_kernel<F32, STEPS, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, low_bytes<F32, STEPS>);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_args(const qmm_adapter_desc* d, const qmm_adapter_args* a) {
    if (a == nullptr) return QMM_ERR_INVALID_ARG;
    if (a->rows < 0 || a->rows > d->max_rows) return QMM_ERR_INVALID_ARG;
    if (a->rows == 0) return QMM_OK;
    const void* const wide[3] = {a->x, a->a, a->b};
    for (const void* p : wide)
        if (p == nullptr || !aligned(p, 16)) return QMM_ERR_INVALID_ARG;
    const size_t size = d->out_dtype == QMM_OUT_F32 ? 4 : 2;
    if (a->y == nullptr || a->out == nullptr || !aligned(a->y, size) || !aligned(a->out, size)) return QMM_ERR_INVALID_ARG;
    if (a->ids == nullptr || !aligned(a->ids, 4) || !aligned(a->scale, 4)) return QMM_ERR_INVALID_ARG;
    if (a->rows > 1) {
        const int64_t strides[3] = {a->x_stride, a->y_stride, a->out_stride}, least[3] = {d->K, d->N, d->N};
        for (int i = 0; i < 3; ++i)
            if (strides[i] < least[i] || strides[i] > (1LL << 40)) return QMM_ERR_INVALID_ARG;
        if (a->x_stride % 8 != 0) return QMM_ERR_INVALID_ARG;
        if (a->y == a->out && a->y_stride != a->out_stride) return QMM_ERR_INVALID_ARG;
    }
    return QMM_OK;
}

class OnDevice {   // makes a plan's device the current one, and at the end of the call the one that was
public:
    explicit OnDevice(int device) {
        int now = 0;
        ok = cudaGetDevice(&now) == cudaSuccess;
        if (ok && now != device) {
            ok = cudaSetDevice(device) == cudaSuccess;
            before_ = now;
        }
    }
    ~OnDevice() {
        if (before_ >= 0) cudaSetDevice(before_);
    }
    OnDevice(const OnDevice&) = delete;
    OnDevice& operator=(const OnDevice&) = delete;
    bool ok;

private:
    int before_ = -1;
};

}  // namespace

}  // namespace qmmk

using namespace qmmk;

extern "C" {

int qmm_adapter_validate_desc(const qmm_adapter_desc* d) {
    if (d == nullptr) return QMM_ERR_INVALID_ARG;
    if (d->K < 1 || d->N < 1 || d->rank < 1 || d->adapters < 1 || d->max_rows < 1) return QMM_ERR_INVALID_ARG;
    if (d->K > (1LL << 30) || d->N > (1LL << 30) || d->max_rows > QMM_ADAPTER_MAX_ROWS) return QMM_ERR_INVALID_ARG;
    if (d->out_dtype != QMM_OUT_F32 && d->out_dtype != QMM_OUT_BF16) return QMM_ERR_INVALID_ARG;
    if (d->K % 64 != 0 || d->rank % 8 != 0 || d->rank > QMM_ADAPTER_MAX_RANK) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

size_t qmm_adapter_workspace_bytes(const qmm_adapter_desc* d) {
    if (qmm_adapter_validate_desc(d) != QMM_OK) return 0;
    return kErrBytes + static_cast<size_t>(d->max_rows) * d->rank * terms_of(d->out_dtype) * sizeof(uint16_t);
}

int qmm_adapter_plan(qmm_adapter_plan_t** plan, const qmm_adapter_desc* d, void* workspace, size_t ws_bytes) {
    if (plan == nullptr) return QMM_ERR_INVALID_ARG;
    *plan = nullptr;
    const int v = qmm_adapter_validate_desc(d);
    if (v != QMM_OK) return v;
    const size_t need = qmm_adapter_workspace_bytes(d);
    if (workspace != nullptr && (ws_bytes < need || !aligned(workspace, 256))) return QMM_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QMM_ERR_CUDA;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return QMM_ERR_CUDA;
    if (cudaFuncSetAttribute(qmm_adapter_low_kernel<2>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(qmm_adapter_low_kernel<3>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return QMM_ERR_CUDA;
    if (configure_out<true, 1>() != cudaSuccess || configure_out<true, 2>() != cudaSuccess || configure_out<true, 4>() != cudaSuccess ||
        configure_out<false, 4>() != cudaSuccess)
        return QMM_ERR_CUDA;
    struct qmm_adapter_plan* p = new (std::nothrow) struct qmm_adapter_plan();
    if (p == nullptr) return QMM_ERR_ALLOC;
    p->d = *d;
    p->device = dev;
    p->num_sms = sms;
    p->owns_ws = workspace == nullptr;
    void* ws = workspace;
    if (p->owns_ws && cudaMalloc(&ws, need) != cudaSuccess) {
        delete p;
        return QMM_ERR_ALLOC;
    }
    p->ws = static_cast<uint8_t*>(ws);
    if (cudaMemsetAsync(p->ws, 0, kErrBytes, 0) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess) {
        if (p->owns_ws) cudaFree(p->ws);
        delete p;
        return QMM_ERR_CUDA;
    }
    *plan = p;
    return QMM_OK;
}

int qmm_adapter_error(const qmm_adapter_plan_t* p, uint32_t* flags) {
    if (p == nullptr || flags == nullptr) return QMM_ERR_INVALID_ARG;
    uint32_t v = 0;
    const OnDevice on(p->device);
    if (!on.ok) return QMM_ERR_CUDA;
    if (cudaDeviceSynchronize() != cudaSuccess) return QMM_ERR_CUDA;
    if (cudaMemcpy(&v, p->ws, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return QMM_ERR_CUDA;
    if (v != 0 && (cudaMemset(p->ws, 0, sizeof(v)) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess))
        return QMM_ERR_CUDA;
    *flags = v;
    return v == 0 ? QMM_OK : QMM_ERR_INVALID_ARG;
}

void qmm_adapter_destroy(qmm_adapter_plan_t* p) {
    if (p == nullptr) return;
    if (p->owns_ws && p->ws != nullptr) cudaFree(p->ws);
    delete p;
}

int qmm_check_adapter_args(const qmm_adapter_desc* d, const qmm_adapter_args* a) {
    const int v = qmm_adapter_validate_desc(d);
    return v != QMM_OK ? v : check_args(d, a);
}

int qmm_add_adapters(const qmm_adapter_plan_t* p, const qmm_adapter_args* a, void* stream) {
    if (p == nullptr) return QMM_ERR_INVALID_ARG;
    const int chk = check_args(&p->d, a);
    if (chk != QMM_OK) return chk;
    if (a->rows == 0) return QMM_OK;
    const OnDevice on(p->device);
    if (!on.ok) return QMM_ERR_CUDA;
    AdapterParams ap;
    ap.x = static_cast<const uint16_t*>(a->x);
    ap.a = static_cast<const uint16_t*>(a->a);
    ap.b = static_cast<const uint16_t*>(a->b);
    ap.scale = a->scale;
    ap.ids = a->ids;
    ap.y = a->y;
    ap.out = a->out;
    ap.err = reinterpret_cast<uint32_t*>(p->ws);
    ap.low = reinterpret_cast<uint16_t*>(p->ws + kErrBytes);
    ap.low_term = static_cast<int64_t>(p->d.max_rows) * p->d.rank;
    ap.x_stride = a->x_stride;
    ap.y_stride = a->y_stride;
    ap.out_stride = a->out_stride;
    ap.K = p->d.K;
    ap.N = p->d.N;
    ap.rank = p->d.rank;
    ap.adapters = p->d.adapters;
    ap.rows = a->rows;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f32 = p->d.out_dtype == QMM_OUT_F32;
    const int64_t vec = f32 ? 4 : 8;
    const bool wide = aligned(a->y, 16) && aligned(a->out, 16) &&
                      (a->rows == 1 || (a->y_stride % vec == 0 && a->out_stride % vec == 0));
    pthread_mutex_lock(&p->launches);
    cudaError_t e = f32 ? launch_low<3>(ap, p->num_sms, st) : launch_low<2>(ap, p->num_sms, st);
    if (e == cudaSuccess) e = f32 ? launch_out<true>(ap, wide, p->num_sms, st) : launch_out<false>(ap, wide, p->num_sms, st);
    pthread_mutex_unlock(&p->launches);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

}  // extern "C"
