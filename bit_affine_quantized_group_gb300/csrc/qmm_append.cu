// Norms of queries and keys, their rotation, and the append to the paged cache,
// in one pass over the new tokens:
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a c - b s, b c + a s).
// A head is spread over head_dim / 8 lanes with 8 neighbouring elements each
// (16-byte accesses of bfloat16): the mean is a sum over those lanes, and the
// other element of a half-split pair lies rot_dim / 16 lanes away. Everything
// is float32 until the one rounding to bfloat16.
#include <cuda_bf16.h>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_kv.h"

namespace qmmk {

namespace {

constexpr int kAppendWarps = 4;
constexpr int64_t kManyWarps = 152 * 40;   // two rounds of the warps that run at once

// Head vectors that a warp loads before it works on the last ones.
template <bool F32>
constexpr int kAppendSteps = F32 ? 2 : 4;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack_bf16(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
}

// Eight elements as they lie in memory.
template <bool F32>
struct Raw {
    uint4 w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, int64_t elem) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + elem * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) w[i] = __ldg(s + i);
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        if constexpr (F32) {
            x[0] = __uint_as_float(w[0].x), x[1] = __uint_as_float(w[0].y);
            x[2] = __uint_as_float(w[0].z), x[3] = __uint_as_float(w[0].w);
            x[4] = __uint_as_float(w[1].x), x[5] = __uint_as_float(w[1].y);
            x[6] = __uint_as_float(w[1].z), x[7] = __uint_as_float(w[1].w);
        } else {
            unpack_bf16(w[0].x, x[0], x[1]);
            unpack_bf16(w[0].y, x[2], x[3]);
            unpack_bf16(w[0].z, x[4], x[5]);
            unpack_bf16(w[0].w, x[6], x[7]);
        }
    }
};

// One warp takes `span` heads of one token, kSteps vectors of 32 / (D / 8) heads at a time: position, page and rotation are
// looked up once for all of them, and the next vectors are on their way while it works on the last.
template <int D, bool F32>
__global__ void __launch_bounds__(32 * kAppendWarps) qmm_append_kernel(const __grid_constant__ AppendParams p, int span) {
    constexpr int kLanes = D / 8;
    constexpr int kHeads = 32 / kLanes;
    constexpr int kSteps = kAppendSteps<F32>;
    const int lane = threadIdx.x & 31;
    const int heads = p.q_heads + 2 * p.kv_heads;
    const int per_token = (heads + span - 1) / span;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int token = static_cast<int>(unit / per_token);
    const int h0 = static_cast<int>(unit - static_cast<int64_t>(token) * per_token) * span;
    const int h1 = h0 + span < heads ? h0 + span : heads;
    const int e = (lane % kLanes) * 8;   // this lane's elements of a head
    griddep_launch_dependents();
    griddep_wait();
    if (token >= p.tokens) return;

    Raw<F32> next[kSteps];
    auto load = [&](int h) {   // the vectors from head h on
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int hd = h + i * kHeads + lane / kLanes;
            if (hd >= h1) continue;
            const int kind = hd < p.q_heads ? 0 : hd < p.q_heads + p.kv_heads ? 1 : 2;
            const int hk = kind == 0 ? hd : hd - p.q_heads - (kind - 1) * p.kv_heads;
            next[i].load(p.in[kind], token * p.in_stride[kind] + static_cast<int64_t>(hk) * D + e);
        }
    };
    load(h0);

    const int seq = token / p.rows;
    const int pos = p.lengths[seq] - p.rows + (token - seq * p.rows);
    const bool live = pos >= 0;

    // the cache slot
    int64_t k_at = 0, v_at = 0;
    bool store = live;
    if (live) {
        const int slot = pos & ((1 << p.page_shift) - 1);
        const int index = pos >> p.page_shift;
        if (index >= p.max_pages) {
            if (lane == 0) atomicOr(p.err, QMM_KV_BAD_LENGTH);
            store = false;
        } else {
            const int64_t page = p.page_table[static_cast<int64_t>(seq) * p.max_pages + index];
            if (page < 0 || page >= p.num_pages) {
                if (lane == 0) atomicOr(p.err, QMM_KV_BAD_PAGE);
                store = false;
            } else {
                k_at = page * p.k.page + slot * p.k.slot;
                v_at = page * p.v.page + slot * p.v.slot;
            }
        }
    }

    // this lane's cosines and sines: element pairs (e + j, e + j +- rot/2), or (2i, 2i + 1)
    const int half = p.rot_dim >> 1;
    const bool turns = e < p.rot_dim;
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
    bool rotate = p.rot_dim > 0 && live;
    if (rotate) {
        const int at = p.positions != nullptr ? p.positions[token] : pos;
        if (at < 0 || at >= p.rope_len) {
            if (lane == 0) atomicOr(p.err, QMM_KV_BAD_POSITION);
            rotate = false;
        } else if (turns) {
            const float* row = p.rope + static_cast<int64_t>(at) * p.rot_dim;
            if (p.interleaved) {
                const float4 cc = *reinterpret_cast<const float4*>(row + e / 2);
                const float4 ss = *reinterpret_cast<const float4*>(row + half + e / 2);
                c[0] = c[1] = cc.x, c[2] = c[3] = cc.y, c[4] = c[5] = cc.z, c[6] = c[7] = cc.w;
                s[0] = -ss.x, s[1] = ss.x, s[2] = -ss.y, s[3] = ss.y;
                s[4] = -ss.z, s[5] = ss.z, s[6] = -ss.w, s[7] = ss.w;
            } else {
                const int i0 = e < half ? e : e - half;
                const float sign = e < half ? -1.0f : 1.0f;
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const float4 cc = *reinterpret_cast<const float4*>(row + i0 + j);
                    const float4 ss = *reinterpret_cast<const float4*>(row + half + i0 + j);
                    c[j] = cc.x, c[j + 1] = cc.y, c[j + 2] = cc.z, c[j + 3] = cc.w;
                    s[j] = sign * ss.x, s[j + 1] = sign * ss.y, s[j + 2] = sign * ss.z, s[j + 3] = sign * ss.w;
                }
            }
        }
    }
    const int other = !turns ? lane : e < half ? lane + half / 8 : lane - half / 8;

#pragma unroll 1
    for (int h = h0; h < h1; h += kSteps * kHeads) {
        Raw<F32> now[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) now[i] = next[i];
        load(h + kSteps * kHeads);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int hd = h + i * kHeads + lane / kLanes;
            const bool in = hd < h1;
            const int kind = hd < p.q_heads ? 0 : hd < p.q_heads + p.kv_heads ? 1 : 2;
            const int hk = kind == 0 ? hd : hd - p.q_heads - (kind - 1) * p.kv_heads;
            float y[8];
            now[i].values(y);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(y[j], y[j], sum);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            const float* weight = kind < 2 ? p.weight[kind] : nullptr;
            if (weight != nullptr) {
                const float inv = rsqrtf(sum * (1.0f / D) + p.eps);
                const float4 a = __ldg(reinterpret_cast<const float4*>(weight + e));
                const float4 b = __ldg(reinterpret_cast<const float4*>(weight + e + 4));
                y[0] *= inv * a.x, y[1] *= inv * a.y, y[2] *= inv * a.z, y[3] *= inv * a.w;
                y[4] *= inv * b.x, y[5] *= inv * b.y, y[6] *= inv * b.z, y[7] *= inv * b.w;
            }
            if (rotate) {
                float z[8];
                if (p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] = y[j ^ 1];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] = __shfl_sync(0xFFFFFFFFu, y[j], other);
                }
                if (turns && kind < 2) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = fmaf(y[j], c[j], z[j] * s[j]);
                }
            }
            uint4 w = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
            uint16_t* dst = nullptr;
            if (kind == 0) {
                if (!live) w = make_uint4(0u, 0u, 0u, 0u);
                dst = p.q_out + token * p.q_out_stride + static_cast<int64_t>(hk) * D + e;
            } else if (store) {
                dst = kind == 1 ? p.k.base + k_at + hk * p.k.head + e : p.v.base + v_at + hk * p.v.head + e;
            }
            if (in && dst != nullptr) *reinterpret_cast<uint4*>(dst) = w;
        }
    }
}

template <int D, bool F32>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
    // few tokens: a warp for every load in flight; many: equal parts of a token, up to all of it
    constexpr int kPerLoad = 32 / (D / 8) * kAppendSteps<F32>;
    const int heads = p.q_heads + 2 * p.kv_heads;
    const int64_t loads = (heads + kPerLoad - 1) / kPerLoad;
    int64_t each = p.tokens * loads / kManyWarps;
    each = each < 1 ? 1 : each > loads ? loads : each;
    const int64_t parts = (loads + each - 1) / each;
    const int span = static_cast<int>((loads + parts - 1) / parts) * kPerLoad;
    const int64_t per_token = (heads + span - 1) / span;
    const int64_t blocks = (p.tokens * per_token + kAppendWarps - 1) / kAppendWarps;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(32 * kAppendWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qmm_append_kernel<D, F32>, p, span);
}

}  // namespace

cudaError_t launch_append(int head_dim, bool in_f32, const AppendParams& p, cudaStream_t stream) {
    if (head_dim == 64) return in_f32 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
    if (head_dim == 128) return in_f32 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
    return in_f32 ? launch<256, true>(p, stream) : launch<256, false>(p, stream);
}

}  // namespace qmmk
