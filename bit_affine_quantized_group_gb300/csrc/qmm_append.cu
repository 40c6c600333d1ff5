// Norms of queries and keys, their rotation, and the append to the paged cache,
// in one pass over the new tokens:
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a c - b s, b c + a s).
// A head is spread over head_dim / 8 lanes with eight elements each, four a and
// the four b that they turn with, so that a pair never leaves its lane: where
// the halves of the rotated part turn with one another, a lane has four
// neighbours of each half. The mean is a sum over the lanes. Everything is
// float32 until the one rounding to bfloat16.
//
// The bound of many tokens is the bytes, but instructions are close to it: 4 x
// 2048 tokens of 48 heads of 128 take 35.1 us, 5.8 TB/s, where pairs that met by
// shuffles, single float32 operations and addresses computed for every vector
// took 45 at 66 % of the issue slots. Few tokens are bound by latency (2.2 us for
// one), and a warp takes only as many heads as it can have in flight.
//
// For a cache of codes a head's float32 values pass through shared memory, after
// which a lane has eight neighbours and eight lanes a group of 64, whose least
// and largest they find by shuffles:
//   b = f16(lo),  s = f16((hi - lo) / top),  c = round((x - b) (1 / s)).
// The same 4 x 2048 tokens: 40 us, bound by instructions (34.2 M of warps, 28.5 M
// for the bfloat16 cache), of which spills and values' trip through shared memory,
// as if they were to be rotated, are a part, with seven CTAs on an SM.
#include <cuda_bf16.h>

#include <type_traits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_kv.h"

namespace qmmk {

namespace {

constexpr int kAppendWarps = 4;
// Parts of tokens that are worth it: a few more than the warps that run at once. (Three times as many took a
// fifteenth longer for the 4 x 2048 tokens, for what a warp looks up for a token outweighs a fuller last round.)
constexpr int64_t kManyWarps = 152 * 40;

// Head vectors that a warp loads before it works on the last ones: with one or four the 4 x 2048 tokens took about a tenth
// longer: less in flight, or fewer warps on an SM.
constexpr int kAppendSteps = 2;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack_bf16(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
}

// Two float32 operations at once.
__device__ __forceinline__ uint64_t bits2(const float2& v) { return *reinterpret_cast<const uint64_t*>(&v); }
__device__ __forceinline__ float2 mul2(const float2& a, const float2& b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return *reinterpret_cast<const float2*>(&d);
}

// A lane's elements: a[j] turns with b[j].
struct Pairs {
    float2 a[2], b[2];
};

// Float32 elements x (four from e0 on, or the first of eight) and y: pairs of neighbours (NEAR), or of x and y.
template <bool NEAR>
__device__ __forceinline__ Pairs pairs_of(const float4& x, const float4& y) {
    Pairs v;
    if constexpr (NEAR) {
        v.a[0] = make_float2(x.x, x.z), v.b[0] = make_float2(x.y, x.w);
        v.a[1] = make_float2(y.x, y.z), v.b[1] = make_float2(y.y, y.w);
    } else {
        v.a[0] = make_float2(x.x, x.y), v.a[1] = make_float2(x.z, x.w);
        v.b[0] = make_float2(y.x, y.y), v.b[1] = make_float2(y.z, y.w);
    }
    return v;
}

// A lane's eight elements as they lie in memory.
template <bool F32, bool NEAR>
struct Raw {
    uint4 w[F32 ? 2 : 1];
    // the elements at `first`, and four more at `second` bytes from there (plain loads: the kernel before may still write them when
    // this one starts, which __ldg does not allow)
    __device__ __forceinline__ void load(const uint8_t* first, int second) {
        if constexpr (F32) {
            w[0] = *reinterpret_cast<const uint4*>(first);
            w[1] = *reinterpret_cast<const uint4*>(first + second);
        } else if constexpr (NEAR) {
            w[0] = *reinterpret_cast<const uint4*>(first);
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(first);
            const uint2 y = *reinterpret_cast<const uint2*>(first + second);
            w[0] = make_uint4(x.x, x.y, y.x, y.y);
        }
    }
    __device__ __forceinline__ Pairs values() const {
        float4 x, y;
        if constexpr (F32) {
            x = make_float4(__uint_as_float(w[0].x), __uint_as_float(w[0].y), __uint_as_float(w[0].z), __uint_as_float(w[0].w));
            y = make_float4(__uint_as_float(w[1].x), __uint_as_float(w[1].y), __uint_as_float(w[1].z), __uint_as_float(w[1].w));
        } else {
            unpack_bf16(w[0].x, x.x, x.y);
            unpack_bf16(w[0].y, x.z, x.w);
            unpack_bf16(w[0].z, y.x, y.y);
            unpack_bf16(w[0].w, y.z, y.w);
        }
        return pairs_of<NEAR>(x, y);
    }
};

template <bool NEAR>
__device__ __forceinline__ void store_pairs(uint16_t* dst, int second, const Pairs& v) {
    if constexpr (NEAR) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(v.a[0].x, v.b[0].x), pack_bf16(v.a[0].y, v.b[0].y),
                                                    pack_bf16(v.a[1].x, v.b[1].x), pack_bf16(v.a[1].y, v.b[1].y));
    } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v.a[0].x, v.a[0].y), pack_bf16(v.a[1].x, v.a[1].y));
        *reinterpret_cast<uint2*>(dst + second) = make_uint2(pack_bf16(v.b[0].x, v.b[0].y), pack_bf16(v.b[1].x, v.b[1].y));
    }
}

// (a or b is NaN: so is the result)
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Eight neighbouring values of a head as codes, of 8 or 4 bits in 8 or 4 bytes. Whole warps call it, the lanes of a group of
// 64 together; `affine` gets their scale and bias. False: a value was not finite.
template <int BITS>
__device__ __forceinline__ bool quantise(float (&x)[8], uint32_t (&codes)[BITS / 4], uint32_t& affine) {
    constexpr float kTop = (1 << BITS) - 1, kLargest = QMM_KVQ_LARGEST;
    auto limits = [&](float& lo, float& hi) {
        lo = hi = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = min_nan(lo, x[i]);
            hi = max_nan(hi, x[i]);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
        }
    };
    float lo, hi;
    limits(lo, hi);
    bool finite = true;
    if (__any_sync(0xFFFFFFFFu, !(lo >= -kLargest && hi <= kLargest))) {   // (NaN among them)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            finite &= fabsf(x[i]) < INFINITY;
            x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -kLargest), kLargest) : 0.0f;
        }
        limits(lo, hi);
    }
    const __half scale = __float2half_rn(__fdiv_rn(hi - lo, kTop)), bias = __float2half_rn(lo);
    const float s = __half2float(scale), b = __half2float(bias);
    const float inverse = s > 0.0f ? __frcp_rn(s) : 0.0f;
    affine = static_cast<uint32_t>(__half_as_ushort(scale)) | static_cast<uint32_t>(__half_as_ushort(bias)) << 16;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float f[2];
        add_x2(f[0], f[1], x[i], x[i + 1], -b, -b);
        mul_x2(f[0], f[1], f[0], f[1], inverse, inverse);
        f[0] = fminf(fmaxf(f[0], 0.0f), kTop), f[1] = fminf(fmaxf(f[1], 0.0f), kTop);
        // the sums' last bits are the whole numbers, rounded to the nearest, ties to even
        add_x2(f[0], f[1], f[0], f[1], 0x1p23f, 0x1p23f);
        c[i] = __float_as_uint(f[0]), c[i + 1] = __float_as_uint(f[1]);
    }
    if constexpr (BITS == 8) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            codes[k] = __byte_perm(__byte_perm(c[4 * k], c[4 * k + 1], 0x0040), __byte_perm(c[4 * k + 2], c[4 * k + 3], 0x0040),
                                   0x5410);
    } else {
        uint32_t two[4];   // (the sums' upper bits are shifted out, or masked)
#pragma unroll
        for (int k = 0; k < 4; ++k) two[k] = (c[2 * k] & 15u) | ((c[2 * k + 1] & 15u) << 4);
        codes[0] = __byte_perm(__byte_perm(two[0], two[1], 0x0040), __byte_perm(two[2], two[3], 0x0040), 0x5410);
    }
    return finite;
}

// One warp takes `span` heads of one token, kSteps vectors of 32 / (D / 8) heads at a time: position, page and rotation are
// looked up once for all of them, and the next vectors are on their way while it works on the last.
// BITS: of a cache of codes; 16 for one of bfloat16.
template <int D, bool F32, bool NEAR, int BITS>
__device__ __forceinline__ void append(const AppendParams& p, int span) {
    constexpr int kLanes = D / 8;
    constexpr int kHeads = 32 / kLanes;
    constexpr int kSteps = kAppendSteps;
    constexpr int kSize = F32 ? 4 : 2;
    __shared__ __align__(16) float s_heads[BITS != 16 && !NEAR ? kAppendWarps * kHeads * D : 4];
    float* const head_values = s_heads + (BITS != 16 && !NEAR ? (threadIdx.x >> 5) * kHeads * D : 0);
    const int lane = threadIdx.x & 31;
    const int heads = p.q_heads + 2 * p.kv_heads, qk_heads = p.q_heads + p.kv_heads;
    const int per_token = (heads + span - 1) / span;
    // (32 bits: tokens have 384 bytes or more for each part, so that the memory holds fewer than 2^30 parts)
    const uint32_t unit = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int token = static_cast<int>(unit / static_cast<uint32_t>(per_token));
    const int h0 = static_cast<int>(unit - static_cast<uint32_t>(token) * per_token) * span;
    const int h1 = h0 + span < heads ? h0 + span : heads;
    // this lane's elements of a head: four from e0 on, and four `second` elements later
    const int l = lane % kLanes;
    const bool turns = l < p.rot_dim / 8;
    const bool split = !NEAR && turns;
    const int e0 = split ? 4 * l : 8 * l, second = split ? p.rot_dim / 2 : 4;
    griddep_launch_dependents();
    griddep_wait();
    if (token >= p.tokens) return;

    // rows of the token, as if each held all heads
    const uint8_t* src[3];
#pragma unroll
    for (int k = 0; k < 3; ++k)
        src[k] = static_cast<const uint8_t*>(p.in[k]) +
                 (token * p.in_stride[k] - (k == 0 ? 0 : k == 1 ? p.q_heads : qk_heads) * D + e0) * kSize;
    Raw<F32, NEAR> next[kSteps];
    auto load = [&](int h) {   // the vectors from head h on
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int hd = h + i * kHeads + lane / kLanes;
            if (hd < h1) next[i].load((hd < p.q_heads ? src[0] : hd < qk_heads ? src[1] : src[2]) + hd * (D * kSize), second * kSize);
        }
    };
    load(h0);

    const int seq = token / p.rows;
    const int pos = max(p.lengths[seq], 0) - p.rows + (token - seq * p.rows);   // (no length wraps)
    if (pos < 0) {   // a token before the sequence's first: its queries are zero
        for (int hd = h0 + lane / kLanes; hd < h1 && hd < p.q_heads; hd += kHeads)
            *reinterpret_cast<uint4*>(p.q_out + token * p.q_out_stride + static_cast<int64_t>(hd) * D + 8 * l) =
                make_uint4(0u, 0u, 0u, 0u);
        return;
    }

    // where head 0 would lie, and from head to head (codes: of this lane's eight neighbours, and their group's pair)
    uint8_t *code[2] = {}, *pair[2] = {};
    const int64_t code_step[2] = {p.k.head, p.v.head}, pair_step[2] = {p.ka.head, p.va.head};
    uint16_t* dst[3] = {p.q_out + token * p.q_out_stride + e0, nullptr, nullptr};
    const int64_t step[3] = {D, p.k.head, p.v.head};
    bool store = false;
    const int slot = pos & ((1 << p.page_shift) - 1), index = pos >> p.page_shift;
    if (index >= p.max_pages) {
        if (lane == 0) atomicOr(p.err, QMM_KV_BAD_LENGTH);
    } else {
        const int64_t page = p.page_table[static_cast<int64_t>(seq) * p.max_pages + index];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) atomicOr(p.err, QMM_KV_BAD_PAGE);
        } else {
            if constexpr (BITS == 16) {
                dst[1] = p.k.base + page * p.k.page + slot * p.k.slot - p.q_heads * p.k.head + e0;
                dst[2] = p.v.base + page * p.v.page + slot * p.v.slot - qk_heads * p.v.head + e0;
            } else {   // strides of bytes, and of pairs of 4 bytes
                code[0] = reinterpret_cast<uint8_t*>(p.k.base) + page * p.k.page + slot * p.k.slot - p.q_heads * p.k.head + l * BITS;
                code[1] = reinterpret_cast<uint8_t*>(p.v.base) + page * p.v.page + slot * p.v.slot - qk_heads * p.v.head + l * BITS;
                pair[0] = reinterpret_cast<uint8_t*>(p.ka.base) +
                          4 * (page * p.ka.page + slot * p.ka.slot - p.q_heads * p.ka.head + l / 8);
                pair[1] = reinterpret_cast<uint8_t*>(p.va.base) +
                          4 * (page * p.va.page + slot * p.va.slot - qk_heads * p.va.head + l / 8);
            }
            store = true;
        }
    }

    // this lane's cosines and sines
    float2 c[2], s[2], neg[2];
    bool rotate = p.rot_dim > 0;
    if (rotate) {
        const int at = p.positions != nullptr ? p.positions[token] : pos;
        if (at < 0 || at >= p.rope_len) {
            if (lane == 0) atomicOr(p.err, QMM_KV_BAD_POSITION);
            rotate = false;
        } else if (turns) {
            const float* row = p.rope + static_cast<int64_t>(at) * p.rot_dim + 4 * l;
            const float4 cc = *reinterpret_cast<const float4*>(row), ss = *reinterpret_cast<const float4*>(row + p.rot_dim / 2);
            c[0] = make_float2(cc.x, cc.y), c[1] = make_float2(cc.z, cc.w);
            s[0] = make_float2(ss.x, ss.y), s[1] = make_float2(ss.z, ss.w);
            neg[0] = make_float2(-ss.x, -ss.y), neg[1] = make_float2(-ss.z, -ss.w);
        }
    }
    rotate = rotate && turns;

#pragma unroll 1
    for (int h = h0; h < h1; h += kSteps * kHeads) {
        Raw<F32, NEAR> now[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) now[i] = next[i];
        load(h + kSteps * kHeads);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int first = h + i * kHeads, hd = first + lane / kLanes;   // the first lane's head, and this one's
            Pairs y = now[i].values();
            if (first < qk_heads) {   // else nothing but values
                float2 sq = mul2(y.a[0], y.a[0]);
                sq = fma2(y.a[1], y.a[1], sq);
                sq = fma2(y.b[0], y.b[0], sq);
                sq = fma2(y.b[1], y.b[1], sq);
                float sum = sq.x + sq.y;
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                if (hd < qk_heads) {
                    const float* weight = hd < p.q_heads ? p.weight[0] : p.weight[1];
                    if (weight != nullptr) {
                        const float inv = rsqrtf(sum * (1.0f / D) + p.eps);
                        const Pairs w = pairs_of<NEAR>(__ldg(reinterpret_cast<const float4*>(weight + e0)),
                                                       __ldg(reinterpret_cast<const float4*>(weight + e0 + second)));
                        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            y.a[j] = mul2(y.a[j], mul2(w.a[j], inv2));
                            y.b[j] = mul2(y.b[j], mul2(w.b[j], inv2));
                        }
                    }
                    if (rotate) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float2 a = fma2(y.a[j], c[j], mul2(y.b[j], neg[j]));
                            y.b[j] = fma2(y.b[j], c[j], mul2(y.a[j], s[j]));
                            y.a[j] = a;
                        }
                    }
                }
            }
            const int kind = hd < p.q_heads ? 0 : hd < qk_heads ? 1 : 2;
            if constexpr (BITS != 16) {
                if (first + kHeads > p.q_heads && first < h1) {   // (the whole warp) keys or values among the heads
                    float x[8];
                    if constexpr (NEAR) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            x[4 * j] = y.a[j].x, x[4 * j + 1] = y.b[j].x, x[4 * j + 2] = y.a[j].y, x[4 * j + 3] = y.b[j].y;
                    } else {
                        float* const own = head_values + (lane / kLanes) * D;
                        __syncwarp();
                        *reinterpret_cast<float4*>(own + e0) = make_float4(y.a[0].x, y.a[0].y, y.a[1].x, y.a[1].y);
                        *reinterpret_cast<float4*>(own + e0 + second) = make_float4(y.b[0].x, y.b[0].y, y.b[1].x, y.b[1].y);
                        __syncwarp();
                        const float4 u = *reinterpret_cast<const float4*>(own + 8 * l), w = *reinterpret_cast<const float4*>(own + 8 * l + 4);
                        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
                    }
                    uint32_t c[BITS / 4], affine;
                    const bool finite = quantise<BITS>(x, c, affine);
                    if (kind != 0 && hd < h1 && store) {
                        uint8_t* const to = (kind == 1 ? code[0] : code[1]) + hd * (kind == 1 ? code_step[0] : code_step[1]);
                        if constexpr (BITS == 8) *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
                        else *reinterpret_cast<uint32_t*>(to) = c[0];
                        if (l % 8 == 0)
                            *reinterpret_cast<uint32_t*>((kind == 1 ? pair[0] : pair[1]) +
                                                         4 * hd * (kind == 1 ? pair_step[0] : pair_step[1])) = affine;
                        if (!finite) atomicOr(p.err, QMM_KV_NOT_FINITE);
                    }
                }
                if (hd < h1 && kind == 0) store_pairs<NEAR>(dst[0] + hd * step[0], second, y);
            } else if (hd < h1 && (kind == 0 || store)) {
                uint16_t* const base = kind == 0 ? dst[0] : kind == 1 ? dst[1] : dst[2];
                store_pairs<NEAR>(base + hd * (kind == 0 ? step[0] : kind == 1 ? step[1] : step[2]), second, y);
            }
        }
    }
}

template <int D, bool F32, bool NEAR>
__global__ void __launch_bounds__(32 * kAppendWarps) qmm_append_kernel(const __grid_constant__ AppendParams p, int span) {
    append<D, F32, NEAR, 16>(p, span);
}

// Registers are held to seven CTAs an SM, though all but four kernels spill 24 to 108 bytes then: 4 x 2048 tokens 40 us, with six
// 44 and with eight 42.
template <int D, bool F32, bool NEAR, int BITS>
__global__ void __launch_bounds__(32 * kAppendWarps, 7) qmm_append_codes_kernel(const __grid_constant__ AppendParams p, int span) {
    append<D, F32, NEAR, BITS>(p, span);
}

template <int D, bool F32, bool NEAR, int BITS>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
    // few tokens: a warp for every load in flight; many: equal parts of a token, up to all of it
    constexpr int kPerLoad = 32 / (D / 8) * kAppendSteps;
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
    if constexpr (BITS == 16) return cudaLaunchKernelEx(&cfg, qmm_append_kernel<D, F32, NEAR>, p, span);
    else return cudaLaunchKernelEx(&cfg, qmm_append_codes_kernel<D, F32, NEAR, BITS>, p, span);
}

}  // namespace

cudaError_t launch_append(int head_dim, bool in_f32, int bits, const AppendParams& p, cudaStream_t stream) {
    auto with = [&](auto f32, auto near, auto of) -> cudaError_t {
        constexpr bool F32 = decltype(f32)::value, NEAR = decltype(near)::value;
        constexpr int BITS = decltype(of)::value;
        if (head_dim == 64) return launch<64, F32, NEAR, BITS>(p, stream);
        if (head_dim == 128) return launch<128, F32, NEAR, BITS>(p, stream);
        return launch<256, F32, NEAR, BITS>(p, stream);
    };
    const std::true_type yes;
    const std::false_type no;
    auto of_bits = [&](auto of) -> cudaError_t {
        if (in_f32) return p.interleaved ? with(yes, yes, of) : with(yes, no, of);
        return p.interleaved ? with(no, yes, of) : with(no, no, of);
    };
    if (bits == 8) return of_bits(std::integral_constant<int, 8>());
    if (bits == 4) return of_bits(std::integral_constant<int, 4>());
    return of_bits(std::integral_constant<int, 16>());
}

}  // namespace qmmk
