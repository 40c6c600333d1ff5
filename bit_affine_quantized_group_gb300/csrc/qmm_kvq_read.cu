// Reads a cache of codes back into dense keys and values: s c + b, one fused
// multiply-add, of every position of a sequence from its first row on.
//
// The bound is the bytes: bits/8 + 4/64 of an element in, 2 or 4 out, where
// instructions are few enough: with indexes and pages looked up for every 16
// bytes they were 174 for those, 81 % of the issue slots at 4.5 TB/s. A thread
// has the same 16 bytes of four positions of a page; neighbours write neighbours.
// 16 sequences of up to 8191 positions of 8 heads of 128, 8 bits to bfloat16: 67.2
// us, 6.2 TB/s, 4 bits 65.8 (51.5 of bytes); two of 100 positions: 2.2 us, a launch.
// The loads are plain ones, for the append before may still be writing when this
// kernel starts; held to the registers of eight CTAs an SM, without which they took
// 72.4 us. (66.6 with loads of memory that nobody writes, which it is not.)
#include <cuda_bf16.h>

#include <type_traits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_kv.h"

namespace qmmk {

namespace {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 4;    // positions of a thread: neighbours from a multiple of four on

// 16 bytes of values from their codes and the group's scale and bias.
template <bool F32, int BITS, class Word>
__device__ __forceinline__ uint4 values_of(const Word& word, uint32_t pair) {
    constexpr int kElems = F32 ? 4 : 8;
    const float2 sb = __half22float2(*reinterpret_cast<const __half2*>(&pair));
    uint32_t w[2];
    if constexpr (sizeof(Word) == 8) w[0] = word.x, w[1] = word.y;
    else w[0] = w[1] = word;
    float v[kElems];
#pragma unroll
    for (int k = 0; k < kElems; k += 2) {   // 2^23 + c, less 2^23
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int bit = (k + j) * BITS;
            if constexpr (BITS == 8) f[j] = __uint_as_float(__byte_perm(w[bit / 32], 0x4B000000u, 0x7440 + bit % 32 / 8));
            else f[j] = __uint_as_float(((w[bit / 32] >> (bit % 32)) & 15u) | 0x4B000000u);
        }
        add_x2(f[0], f[1], f[0], f[1], -0x1p23f, -0x1p23f);
        fma_x2(v[k], v[k + 1], f[0], f[1], sb.x, sb.x, sb.y, sb.y);
    }
    if constexpr (F32) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    } else {
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            b[k] = *reinterpret_cast<const uint32_t*>(&two);
        }
        return make_uint4(b[0], b[1], b[2], b[3]);
    }
}

template <int D, bool F32, int BITS>
__global__ void __launch_bounds__(kReadThreads, 8) qmm_kvq_read_kernel(const __grid_constant__ ReadParams p, uint32_t tiles) {
    constexpr int kElems = F32 ? 4 : 8;                // of an output of 16 bytes
    constexpr int kUnits = D / kElems;                 // of a head
    constexpr int kBytes = kElems * BITS / 8;          // of their codes: 2, 4 or 8
    using Word = std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>;
    const uint32_t tile = blockIdx.x % tiles, of = blockIdx.x / tiles;
    const int seq = static_cast<int>(of >> 1), s = static_cast<int>(of & 1);
    griddep_launch_dependents();
    griddep_wait();
    const int given = p.lengths[seq], len = min(given, p.positions);
    const int start = p.starts != nullptr ? p.starts[seq] : 0;
    if (given > p.positions && tile == 0 && threadIdx.x == 0) atomicOr(p.err, QMM_KV_BAD_LENGTH);
    const uint32_t width = p.kv_heads * kUnits;        // units of a position
    const uint32_t u = tile * kReadThreads + threadIdx.x, group = u / width, unit = u - group * width;
    // the thread's positions pos0.., and their rows
    const int64_t pos0 = (static_cast<int64_t>(start) & ~static_cast<int64_t>(kReadRows - 1)) + static_cast<int64_t>(group) * kReadRows;
    const int64_t row0 = pos0 - start;
    if (pos0 + kReadRows <= 0 || pos0 >= len || row0 >= p.rows) return;

    const uint32_t head = unit / kUnits, c = unit % kUnits;
    const KvSide codes = s == 0 ? p.side[0] : p.side[1], pairs = s == 0 ? p.affine[0] : p.affine[1];
    const int32_t* const table = p.page_table + static_cast<int64_t>(seq) * p.max_pages;
    const int32_t at = static_cast<int32_t>(pos0);     // (pos0 is a multiple of four: 0 at least where anything is read)
    const int mask = (1 << p.page_shift) - 1;
    const uint8_t* const from = reinterpret_cast<const uint8_t*>(codes.base) + head * codes.head + c * kBytes;
    const uint32_t* const from_pairs = reinterpret_cast<const uint32_t*>(pairs.base) + head * pairs.head + c * kElems / QMM_KVQ_GROUP;
    auto page_of = [&](int pos) -> int {
        const int page = table[pos >> p.page_shift];
        if (page >= 0 && page < p.num_pages) return page;
        atomicOr(p.err, QMM_KV_BAD_PAGE);
        return -1;
    };
    const int64_t row_stride = (s == 0 ? p.row_stride[0] : p.row_stride[1]) * (F32 ? 4 : 2);
    uint8_t* to = static_cast<uint8_t*>(s == 0 ? p.out[0] : p.out[1]) + (F32 ? 4 : 2) * (seq * (s == 0 ? p.seq_stride[0] : p.seq_stride[1])) +
                  row0 * row_stride + static_cast<int64_t>(unit) * 16;
    const bool together = p.page_shift >= 2;           // the positions lie in one page
    const int page = together ? page_of(at) : -1;
    if (page >= 0 && row0 >= 0 && row0 + kReadRows <= p.rows && pos0 + kReadRows <= len) {
        const int64_t slot = at & mask;
        const uint8_t* src = from + page * codes.page + slot * codes.slot;
        const uint32_t* src_pair = from_pairs + page * pairs.page + slot * pairs.slot;
        Word word[kReadRows];
        uint32_t pair[kReadRows];
#pragma unroll
        for (int i = 0; i < kReadRows; ++i, src += codes.slot, src_pair += pairs.slot) {
            word[i] = *reinterpret_cast<const Word*>(src);
            pair[i] = *src_pair;
        }
#pragma unroll
        for (int i = 0; i < kReadRows; ++i, to += row_stride) *reinterpret_cast<uint4*>(to) = values_of<F32, BITS>(word[i], pair[i]);
        return;
    }
#pragma unroll 1
    for (int i = 0; i < kReadRows; ++i, to += row_stride) {
        if (row0 + i < 0 || row0 + i >= p.rows || pos0 + i >= len) continue;
        const int pg = together ? page : page_of(at + i);
        Word word = Word();
        uint32_t pair = 0;
        if (pg >= 0) {
            const int64_t slot = (at + i) & mask;
            word = *reinterpret_cast<const Word*>(from + pg * codes.page + slot * codes.slot);
            pair = from_pairs[pg * pairs.page + slot * pairs.slot];
        }
        *reinterpret_cast<uint4*>(to) = values_of<F32, BITS>(word, pair);
    }
}

template <int D, bool F32, int BITS>
cudaError_t launch(const ReadParams& p, cudaStream_t stream) {
    // (the first group of four may begin up to three rows before row 0)
    const int64_t groups = (static_cast<int64_t>(p.rows) + 2 * (kReadRows - 1)) / kReadRows;
    const int64_t tiles = (groups * p.kv_heads * (D / (F32 ? 4 : 8)) + kReadThreads - 1) / kReadThreads;
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
