// Codes of a quantized cache in the attention kernels: binary16 numbers from codes, and queries as binary16 numbers.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace qmmk {

namespace {

constexpr uint32_t kHalf1024 = 0x64006400u, kHalf64 = 0x54005400u;   // pairs of binary16 numbers
constexpr float kWeightBits = 15.0f;   // weights are binary16 numbers of up to 2^15, so that those from 2^-29 on keep their bits

__device__ __forceinline__ uint32_t bits_of(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ __half2 half2_of(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ uint32_t pack_f16(float a, float b) { return bits_of(__floats2half2_rn(a, b)); }

__device__ __forceinline__ float sum_f16(uint32_t pair) {
    const float2 v = __half22float2(half2_of(pair));
    return v.x + v.y;
}

// Weights a and b, at least 0, as pairs of binary16 numbers: their upper 11 bits, and the rounded remainders. hi + lo is within
// 2^-21 of a weight, or within 2^-24 where that is more.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
    const float x = __uint_as_float(__float_as_uint(a) & 0xFFFFE000u), y = __uint_as_float(__float_as_uint(b) & 0xFFFFE000u);
    hi = pack_f16(x, y);
    lo = pack_f16(a - x, b - y);
}
// Remainders of 2^-24 at least, where hi is not 0: a remainder of 0 times an infinite value were NaN, where the weight times it
// is infinite.
__device__ __forceinline__ uint32_t some_left(uint32_t hi, uint32_t lo) {
    return bits_of(__hmax2(half2_of(lo), __hmin2(half2_of(hi), half2_of(0x00010001u))));
}

// (x & mask) | bits in one instruction (of two constants the compiler makes two).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
    return d;
}

// The larger magnitude of a pair of bfloat16 numbers, as an integer.
__device__ __forceinline__ uint32_t magnitude(uint32_t w) { return max(w & 0x7FFFu, (w >> 16) & 0x7FFFu); }

// A query row's power of two, which brings its largest magnitude to 2^14..2^15 in binary16 (elements down to 2^-28 of that
// keep all their bits), and what its scores then count in powers of two. That is not 0: masked scores of -infinity were NaN.
struct QuerySize {
    float factor, unit;
    __device__ __forceinline__ QuerySize(uint32_t most, float scale_log2) {
        const int power = min(141 - static_cast<int>(most >> 7), 126);
        factor = __uint_as_float(static_cast<uint32_t>(127 + power) << 23);
        unit = fmaxf(scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - power) << 23), 1e-45f);
    }
    __device__ __forceinline__ uint32_t f16(uint32_t w) const {
        return pack_f16(__uint_as_float(w << 16) * factor, __uint_as_float(w & 0xFFFF0000u) * factor);
    }
};

}  // namespace

}  // namespace qmmk
