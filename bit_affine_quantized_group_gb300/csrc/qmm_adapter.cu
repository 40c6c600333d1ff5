// Low-rank adapters of many requests beside a projection that they share:
//   low[m, :] = scale[i] * x[m, :] A[i]^T,   out[m, :] = y[m, :] + low[m, :] B[i]^T,   i = ids[m].
//
// Both products are m16n8k16 tensor-core products of up to 16 rows of one
// adapter: the rows of a block of 64 are put in the order of their adapters and
// cut into such tiles, which every CTA does for itself. Their bound is bytes: A
// and B of the adapters in use once, x, y and out.
//   - low: the warps of a cluster's CTAs take a tile's 8 columns of rank each,
//     the CTAs slices of K, and add their partial sums through distributed shared
//     memory in the order of the slices.
//   - out: warps take a tile's 32 columns each. low enters as two bfloat16 terms
//     (high + low within 2^-17), which is below what float32 outputs of that many
//     terms are off by; one term would round more than bfloat16 outputs do.
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
constexpr int kStepK = 64;            // elements of x that a lane group loads at once
constexpr size_t kErrBytes = 256;

struct AdapterParams {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scale;
    const int32_t* ids;
    const void* y;
    void* out;
    uint16_t* high;          // [rows, rank] two bfloat16 terms of low
    uint16_t* low;
    uint32_t* err;
    int64_t x_stride, y_stride, out_stride;
    int64_t K, N;
    int32_t rank, adapters, rows;
};

// The rows of a block in the order of their adapters (-1 first), and the tiles of up to 16 of one adapter.
struct Tiles {
    int32_t id[kBlock];      // of the rows as they stand
    uint8_t row[kBlock];     // at each place of the order
    int32_t tile_id[kBlock];
    uint8_t first[kBlock], size[kBlock];   // places of a tile
    uint32_t starts[2];
    int tiles;
};

// By the whole CTA; ids outside -1..adapters-1 count as -1.
__device__ __forceinline__ void find_tiles(const AdapterParams& p, int row0, Tiles& t) {
    const int tid = threadIdx.x, rows = min(kBlock, p.rows - row0);
    int id = -1;
    if (tid < rows) {
        id = p.ids[row0 + tid];
        if (id < -1 || id >= p.adapters) {
            atomicOr(p.err, static_cast<uint32_t>(QMM_ADAPTER_BAD_ID));
            id = -1;
        }
        t.id[tid] = id;
    }
    __syncthreads();
    if (tid < kBlock) {
        int before = 0, same = 0;   // rows of smaller ids, and earlier rows of this one
        if (tid < rows)
            for (int j = 0; j < rows; ++j) {
                const int other = t.id[j];
                before += other < id;
                same += other == id && j < tid;
            }
        const int place = before + same;
        if (tid < rows) t.row[place] = static_cast<uint8_t>(tid);
        // which places begin a tile
        const bool begins = tid < rows && same % kTile == 0;
        if (tid < 2) t.starts[tid] = 0;
        named_barrier(1, kBlock);
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

// v as two bfloat16 terms; an infinity or NaN stands in the first alone.
__device__ __forceinline__ void split(float v, uint16_t& high, uint16_t& low) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    const float f = __bfloat162float(h);
    high = __bfloat16_as_ushort(h);
    low = __bfloat16_as_ushort(__float2bfloat16_rn(fabsf(f) < INFINITY ? v - f : 0.0f));
}

// 16 elements of a lane: the products' four steps of 64 elements of K, of which a lane of a quad takes 16 neighbours.
struct Sixteen {
    uint4 v[2];
    __device__ __forceinline__ void load(const uint16_t* p) {
        v[0] = __ldg(reinterpret_cast<const uint4*>(p));
        v[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void clear() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ uint32_t word(int i) const {
        const uint4& w = v[i >> 2];
        return (i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w;
    }
};

// Grid: clusters of `slices` CTAs; block of rows, then one of `groups` that share its units (a tile's 8 columns of rank).
__global__ void __launch_bounds__(kThreads) qmm_adapter_low_kernel(const __grid_constant__ AdapterParams p, int slices, int groups) {
    extern __shared__ __align__(16) float s_part[];   // [place][rank] of this CTA's slice
    __shared__ Tiles t;
    cg::cluster_group cluster = cg::this_cluster();
    const int slice = static_cast<int>(blockIdx.x % slices), of = static_cast<int>(blockIdx.x / slices);
    const int group = of % groups, row0 = of / groups * kBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, quad = lane & 3;
    griddep_launch_dependents();
    griddep_wait();
    find_tiles(p, row0, t);
    const int columns = p.rank / 8, units = t.tiles * columns;
    const int64_t steps = p.K / kStepK;
    const int64_t k0 = steps * slice / slices * kStepK, k1 = steps * (slice + 1) / slices * kStepK;

    for (int u = group + warp * groups; u < units; u += kWarps * groups) {
        const int tile = u / columns, column = u - tile * columns, id = t.tile_id[tile];
        if (id < 0) continue;
        const int first = t.first[tile], size = t.size[tile];
        const uint16_t* const a = p.a + (static_cast<int64_t>(id) * p.rank + column * 8 + gid) * p.K + quad * 16;
        const uint16_t* x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int place = gid + 8 * h;
            x[h] = p.x + static_cast<int64_t>(row0 + (place < size ? t.row[first + place] : 0)) * p.x_stride + quad * 16;
        }
        const bool in0 = gid < size, in1 = gid + 8 < size;
        float acc[2][4] = {};   // of the even and the odd steps
        for (int64_t k = k0; k < k1; k += kStepK) {
            Sixteen wa, w0, w1;
            wa.load(a + k);
            if (in0) w0.load(x[0] + k);
            else w0.clear();
            if (in1) w1.load(x[1] + k);
            else w1.clear();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t f[4] = {w0.word(2 * i), w1.word(2 * i), w0.word(2 * i + 1), w1.word(2 * i + 1)};
                mma_bf16(acc[i & 1], f, wa.word(2 * i), wa.word(2 * i + 1));
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (gid + 8 * h < size)
                *reinterpret_cast<float2*>(s_part + (first + gid + 8 * h) * p.rank + column * 8 + quad * 2) =
                    make_float2(acc[0][2 * h] + acc[1][2 * h], acc[0][2 * h + 1] + acc[1][2 * h + 1]);
    }
    cluster.sync();
    // each CTA adds up a share of the units: two elements of up to 4 rows a lane
    int mine = 0;
    for (int u = group; u < units; u += groups, ++mine) {
        if (mine % slices != slice || (mine / slices) % kWarps != warp) continue;
        const int tile = u / columns, column = u - tile * columns, id = t.tile_id[tile];
        if (id < 0) continue;
        const int first = t.first[tile], size = t.size[tile];
        const float by = p.scale != nullptr ? p.scale[id] : 1.0f;
        for (int place = gid; place < size; place += 8) {
            float2 sum = make_float2(0.0f, 0.0f);
            for (int i = 0; i < slices; ++i) {
                const float2 v = *reinterpret_cast<const float2*>(cluster.map_shared_rank(s_part, i) +
                                                                  (first + place) * p.rank + column * 8 + quad * 2);
                sum.x += v.x;
                sum.y += v.y;
            }
            uint16_t h[2], l[2];
            split(sum.x * by, h[0], l[0]);
            split(sum.y * by, h[1], l[1]);
            const int64_t at = static_cast<int64_t>(row0 + t.row[first + place]) * p.rank + column * 8 + quad * 2;
            *reinterpret_cast<uint32_t*>(p.high + at) = h[0] | static_cast<uint32_t>(h[1]) << 16;
            *reinterpret_cast<uint32_t*>(p.low + at) = l[0] | static_cast<uint32_t>(l[1]) << 16;
        }
    }
    cluster.sync();   // other CTAs have read this one's sums
}

// Warps take units of a tile's 32 columns: a lane has 8 neighbouring columns of two rows. WIDE: rows of y and out are read and written 16 bytes at a time.
template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads) qmm_adapter_out_kernel(const __grid_constant__ AdapterParams p, int groups) {
    __shared__ Tiles t;
    using T = std::conditional_t<F32, float, uint16_t>;
    const int group = static_cast<int>(blockIdx.x % groups), row0 = static_cast<int>(blockIdx.x / groups) * kBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, quad = lane & 3;
    griddep_launch_dependents();
    griddep_wait();
    find_tiles(p, row0, t);
    const int64_t columns = (p.N + 31) / 32, units = t.tiles * columns;
    const int steps = (p.rank + 15) / 16;
    for (int64_t u = static_cast<int64_t>(group) * kWarps + warp; u < units; u += static_cast<int64_t>(groups) * kWarps) {
        const int tile = static_cast<int>(u / columns);
        const int64_t n0 = (u - tile * columns) * 32;
        const int id = t.tile_id[tile], first = t.first[tile], size = t.size[tile];
        if (id < 0 && p.y == p.out) continue;
        int64_t row[2];
        bool in[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            in[h] = gid + 8 * h < size;
            row[h] = row0 + (in[h] ? t.row[first + gid + 8 * h] : 0);
        }
        float acc[4][4] = {};   // products of 8 columns: n0 + 8 (their lane's quad) + 2 j + {0, 1}
        if (id >= 0) {
            const uint16_t* b[4];
            bool in_b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + 8 * (gid >> 1) + 2 * j + (gid & 1);
                in_b[j] = n < p.N;
                b[j] = p.b + (static_cast<int64_t>(id) * p.N + (in_b[j] ? n : 0)) * p.rank + quad * 4;
            }
            for (int k = 0; k < steps; ++k) {
                const bool in_k = k * 16 + quad * 4 < p.rank;
                uint32_t f[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint2 hi = make_uint2(0u, 0u), lo = make_uint2(0u, 0u);
                    if (in[h] && in_k) {
                        hi = *reinterpret_cast<const uint2*>(p.high + row[h] * p.rank + k * 16 + quad * 4);
                        lo = *reinterpret_cast<const uint2*>(p.low + row[h] * p.rank + k * 16 + quad * 4);
                    }
                    f[0][h] = hi.x, f[0][h + 2] = hi.y, f[1][h] = lo.x, f[1][h + 2] = lo.y;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint2 w = make_uint2(0u, 0u);
                    if (in_b[j] && in_k) w = __ldg(reinterpret_cast<const uint2*>(b[j] + k * 16));
                    mma_bf16(acc[j], f[0], w.x, w.y);
                    mma_bf16(acc[j], f[1], w.x, w.y);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!in[h]) continue;
            const int64_t n = n0 + quad * 8;
            const T* const y = static_cast<const T*>(p.y) + row[h] * p.y_stride + n;
            T* const out = static_cast<T*>(p.out) + row[h] * p.out_stride + n;
            if (WIDE && n + 8 <= p.N) {
                if constexpr (F32) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float4 v = *reinterpret_cast<const float4*>(y + 4 * k);
                        v.x += acc[2 * k][2 * h], v.y += acc[2 * k][2 * h + 1];
                        v.z += acc[2 * k + 1][2 * h], v.w += acc[2 * k + 1][2 * h + 1];
                        *reinterpret_cast<float4*>(out + 4 * k) = v;
                    }
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(y);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t r[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        r[j] = pack_bf16(__uint_as_float(w[j] << 16) + acc[j][2 * h],
                                         __uint_as_float(w[j] & 0xFFFF0000u) + acc[j][2 * h + 1]);
                    *reinterpret_cast<uint4*>(out) = make_uint4(r[0], r[1], r[2], r[3]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (n + j >= p.N) break;
                    const float add = acc[j >> 1][2 * h + (j & 1)];
                    if constexpr (F32) out[j] = y[j] + add;
                    else out[j] = static_cast<uint16_t>(pack_bf16(__uint_as_float(static_cast<uint32_t>(y[j]) << 16) + add, 0.0f));
                }
            }
        }
    }
}

cudaError_t launch_low(const AdapterParams& p, int num_sms, cudaStream_t stream) {
    const int64_t blocks = (p.rows + kBlock - 1) / kBlock;
    const int64_t steps = p.K / kStepK;
    int slices = kSlices;
    while (slices > steps) slices /= 2;
    // units of a block: one for each 8 columns of rank of up to as many tiles as it has rows
    const int64_t units = static_cast<int64_t>(p.rows < kBlock ? p.rows : kBlock) * (p.rank / 8);
    int64_t groups = 2 * num_sms / (blocks * slices);
    const int64_t most = (units + kWarps - 1) / kWarps;
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
    cfg.dynamicSmemBytes = static_cast<size_t>(kBlock) * p.rank * 4;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, qmm_adapter_low_kernel, p, slices, static_cast<int>(groups));
}

template <bool F32, bool WIDE>
cudaError_t launch_out(const AdapterParams& p, int num_sms, cudaStream_t stream) {
    const int64_t blocks = (p.rows + kBlock - 1) / kBlock;
    const int64_t units = (p.rows < kBlock ? p.rows : kBlock) * ((p.N + 31) / 32);
    int64_t groups = (4 * num_sms + blocks - 1) / blocks;
    const int64_t most = (units + kWarps - 1) / kWarps;
    groups = groups > most ? most : groups;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * groups));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qmm_adapter_out_kernel<F32, WIDE>, p, static_cast<int>(groups));
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
    if (d->K % kStepK != 0 || d->rank % 8 != 0 || d->rank > QMM_ADAPTER_MAX_RANK) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

size_t qmm_adapter_workspace_bytes(const qmm_adapter_desc* d) {
    if (qmm_adapter_validate_desc(d) != QMM_OK) return 0;
    return kErrBytes + static_cast<size_t>(d->max_rows) * d->rank * 2 * sizeof(uint16_t);
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
    if (cudaFuncSetAttribute(qmm_adapter_low_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
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
    ap.high = reinterpret_cast<uint16_t*>(p->ws + kErrBytes);
    ap.low = ap.high + static_cast<size_t>(p->d.max_rows) * p->d.rank;
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
    cudaError_t e = launch_low(ap, p->num_sms, st);
    if (e == cudaSuccess) {
        if (f32) e = wide ? launch_out<true, true>(ap, p->num_sms, st) : launch_out<true, false>(ap, p->num_sms, st);
        else e = wide ? launch_out<false, true>(ap, p->num_sms, st) : launch_out<false, false>(ap, p->num_sms, st);
    }
    pthread_mutex_unlock(&p->launches);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

}  // extern "C"
