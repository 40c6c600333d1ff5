// Reads a cache of codes back into dense keys and values: s c + b, one fused
// multiply-add, of every position of a sequence from its first row on.
//
// The bound is the bytes: bits/8 + 4/64 of an element in, 2 or 4 out. A thread
// has four outputs of 16 bytes on their way; neighbours write neighbours.
#include <cuda_bf16.h>

#include <type_traits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_kv.h"

namespace qmmk {

namespace {

constexpr int kReadThreads = 256;
constexpr int kReadSteps = 4;    // outputs of a thread

template <int D, bool F32, int BITS>
__global__ void __launch_bounds__(kReadThreads) qmm_kvq_read_kernel(const __grid_constant__ ReadParams p, uint32_t tiles) {
    constexpr int kElems = F32 ? 4 : 8;                // of an output of 16 bytes
    constexpr int kUnits = D / kElems;                 // of a head
    constexpr int kBytes = kElems * BITS / 8;          // of their codes: 2, 4 or 8
    using Word = std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>;
    const uint32_t tile = blockIdx.x % tiles, of = blockIdx.x / tiles;
    const int seq = static_cast<int>(of >> 1), s = static_cast<int>(of & 1);
    griddep_launch_dependents();
    griddep_wait();
    const int given = p.lengths[seq], len = min(given, p.positions);
    const int64_t start = p.starts != nullptr ? p.starts[seq] : 0;
    if (given > p.positions && tile == 0 && threadIdx.x == 0) atomicOr(p.err, QMM_KV_BAD_LENGTH);
    const uint32_t units = static_cast<uint32_t>(p.rows) * p.kv_heads * kUnits;
    const uint32_t u0 = tile * (kReadThreads * kReadSteps);
    if (start + u0 / (p.kv_heads * kUnits) >= len) return;

    const KvSide codes = s == 0 ? p.side[0] : p.side[1], pairs = s == 0 ? p.affine[0] : p.affine[1];
    const int32_t* const table = p.page_table + static_cast<int64_t>(seq) * p.max_pages;
    uint8_t* const out = static_cast<uint8_t*>(s == 0 ? p.out[0] : p.out[1]) +
                         (F32 ? 4 : 2) * seq * (s == 0 ? p.seq_stride[0] : p.seq_stride[1]);
    const int64_t row_stride = s == 0 ? p.row_stride[0] : p.row_stride[1];
    Word word[kReadSteps];
    uint32_t pair[kReadSteps];
    uint8_t* to[kReadSteps];
#pragma unroll
    for (int i = 0; i < kReadSteps; ++i) {
        const uint32_t u = u0 + i * kReadThreads + threadIdx.x;
        const uint32_t c = u % kUnits, head_row = u / kUnits;
        const uint32_t row = head_row / static_cast<uint32_t>(p.kv_heads), head = head_row - row * p.kv_heads;
        const int64_t pos = start + row;
        to[i] = nullptr;
        if (u >= units || pos < 0 || pos >= len) continue;
        to[i] = out + (F32 ? 4 : 2) * (row * row_stride + static_cast<int64_t>(head) * D) + c * 16;
        const int32_t at = static_cast<int32_t>(pos);
        const int64_t page = table[at >> p.page_shift], slot = at & ((1 << p.page_shift) - 1);
        word[i] = Word();
        pair[i] = 0;
        if (page < 0 || page >= p.num_pages) {
            atomicOr(p.err, QMM_KV_BAD_PAGE);
            continue;
        }
        word[i] = __ldg(reinterpret_cast<const Word*>(reinterpret_cast<const uint8_t*>(codes.base) + page * codes.page +
                                                      head * codes.head + slot * codes.slot + c * kBytes));
        pair[i] = __ldg(reinterpret_cast<const uint32_t*>(pairs.base) + page * pairs.page + head * pairs.head +
                        slot * pairs.slot + c * kElems / QMM_KVQ_GROUP);
    }
#pragma unroll
    for (int i = 0; i < kReadSteps; ++i) {
        if (to[i] == nullptr) continue;
        const float scale = __half2float(__ushort_as_half(static_cast<uint16_t>(pair[i])));
        const float bias = __half2float(__ushort_as_half(static_cast<uint16_t>(pair[i] >> 16)));
        uint32_t w[2];
        if constexpr (kBytes == 8) w[0] = word[i].x, w[1] = word[i].y;
        else w[0] = w[1] = word[i];
        float v[kElems];
#pragma unroll
        for (int k = 0; k < kElems; ++k) {
            const uint32_t code = (w[k * BITS / 32] >> (k * BITS % 32)) & ((1u << BITS) - 1u);
            v[k] = fmaf(static_cast<float>(code), scale, bias);
        }
        uint4 r;
        if constexpr (F32) {
            r = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        } else {
            uint32_t b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                b[k] = *reinterpret_cast<const uint32_t*>(&two);
            }
            r = make_uint4(b[0], b[1], b[2], b[3]);
        }
        *reinterpret_cast<uint4*>(to[i]) = r;
    }
}

template <int D, bool F32, int BITS>
cudaError_t launch(const ReadParams& p, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(p.rows) * p.kv_heads * (D / (F32 ? 4 : 8));
    const int64_t tiles = (units + kReadThreads * kReadSteps - 1) / (kReadThreads * kReadSteps);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * p.seqs * tiles));
    cfg.blockDim = dim3(kReadThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qmm_kvq_read_kernel<D, F32, BITS>, p, static_cast<uint32_t>(tiles));
}

}  // namespace

cudaError_t launch_read(int head_dim, bool out_f32, int bits, const ReadParams& p, cudaStream_t stream) {
    auto with = [&](auto f32, auto of) -> cudaError_t {
        constexpr bool F32 = decltype(f32)::value;
        constexpr int BITS = decltype(of)::value;
        if (head_dim == 64) return launch<64, F32, BITS>(p, stream);
        if (head_dim == 128) return launch<128, F32, BITS>(p, stream);
        return launch<256, F32, BITS>(p, stream);
    };
    const std::integral_constant<int, 8> eight;
    const std::integral_constant<int, 4> four;
    if (bits == 8) return out_f32 ? with(std::true_type(), eight) : with(std::false_type(), eight);
    return out_f32 ? with(std::true_type(), four) : with(std::false_type(), four);
}

}  // namespace qmmk
