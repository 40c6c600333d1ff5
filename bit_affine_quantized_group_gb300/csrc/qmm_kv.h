// Host and device declarations shared by the cache operators (qmm_kv_api.cu,
// qmm_append.cu, qmm_attention.cu): kernel parameters, the attention kernel's
// workspace layout and the launchers. Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace qmmk {

constexpr size_t kKvErrBytes = 256;        // error word at the start of the workspace
constexpr int kAttnMaxCtas = 320;          // largest grid of the attention kernel (2 CTAs on each of 152 SMs, and room)
constexpr size_t kAttnCounterBytes = 4096; // one join counter per CTA
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnTile = 16;              // positions of one warp's step
constexpr int kAttnUnit = kAttnTile * kAttnWarps;

static_assert(kAttnMaxCtas * 4 <= kAttnCounterBytes, "join counters");

// Query rows (tokens x heads of a group) that one CTA holds: one or two 16-row
// MMA tiles a warp. 256-wide heads have registers for one.
constexpr int attn_row_tiles(int head_dim, int rows) { return head_dim < 256 && rows > 16 ? 2 : 1; }

// Strides in elements.
struct KvSide {
    uint16_t* base;
    int64_t page, head, slot;
};

struct AttnParams {
    KvSide k, v;
    const uint16_t* q;
    uint16_t* out;
    const int32_t* page_table;
    const int32_t* lengths;
    float* part;            // [2 * ctas][16 * MT][D] unnormalised outputs of cut heads
    float* part_ml;         // [2 * ctas][16 * MT][2] their maxima (in powers of two) and sums
    uint32_t* counters;     // [ctas] parts that have arrived, by the CTA that a head starts in; left at zero
    uint32_t* err;
    int64_t q_stride, out_stride, num_pages;
    int32_t seqs, rows, group, kv_heads, row_groups, max_pages, page_shift, window, sinks;
    float scale_log2;       // scale * log2(e)
};

struct AppendParams {
    KvSide k, v;
    const void* in[3];      // q, k, v
    int64_t in_stride[3];
    uint16_t* q_out;
    int64_t q_out_stride;
    const float* weight[2]; // q, k
    const float* rope;
    int64_t rope_len;
    const int32_t* lengths;
    const int32_t* positions;
    const int32_t* page_table;
    uint32_t* err;
    int64_t num_pages;
    int32_t tokens, rows, q_heads, kv_heads, max_pages, page_shift, rot_dim, interleaved;
    float eps;
};

struct AttnWorkspace {
    size_t counters, part, part_ml, bytes;   // offsets
};

constexpr AttnWorkspace attn_workspace(int head_dim, int rows) {
    const size_t slots = 2 * static_cast<size_t>(kAttnMaxCtas) * 16 * attn_row_tiles(head_dim, rows);
    AttnWorkspace w{};
    w.counters = kKvErrBytes;
    w.part_ml = w.counters + kAttnCounterBytes;
    w.part = w.part_ml + slots * 2 * sizeof(float);
    w.bytes = w.part + slots * head_dim * sizeof(float);
    return w;
}

cudaError_t configure_attention();
cudaError_t launch_attention(int head_dim, const AttnParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_append(int head_dim, bool in_f32, const AppendParams& p, cudaStream_t stream);

}  // namespace qmmk
