// Host and device declarations shared by the cache operators (qmm_kv_api.cu,
// qmm_append.cu, qmm_attention.cu): kernel parameters, the attention kernel's
// workspace layout and the launchers. Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace qmmk {

constexpr size_t kKvErrBytes = 256;        // error word at the start of the workspace
constexpr int kAttnMaxCtas = 320;          // largest grid of the attention kernel (2 CTAs on each of 152 SMs, and room)
constexpr size_t kAttnCounterBytes = 4096; // two join counters per CTA

static_assert(2 * kAttnMaxCtas * 4 <= kAttnCounterBytes, "join counters");

// Warps that share a key and value tile with 16 query rows (tokens x heads of a
// group) each. A CTA holds 16 rows for each of them.
constexpr int attn_row_warps(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

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
    float* part;            // [2 * ctas][16 * row warps][D] unnormalised outputs of cut heads
    float* part_ml;         // [2 * ctas][16 * row warps][2] their maxima (in powers of two) and sums
    uint32_t* counters;     // [2][kAttnMaxCtas] parts that have arrived, by the CTA that a head, or a run of its
                            // parts, starts in; left at zero
    int4* joins;            // [ctas] for the join kernel: parts, sequence, cache head and first row of the cut head that
                            // begins in a CTA; no parts for none
    uint32_t* err;
    int64_t q_stride, out_stride, num_pages;
    int32_t seqs, rows, group, kv_heads, row_groups, max_pages, page_shift, window, sinks;
    int32_t positions;      // that the page table holds for a sequence
    int32_t group_inverse;  // ceil(2^20 / group): rows (fewer than 1024) divide by the group (64 at most) exactly
    int32_t min_unit;
    uint32_t query_sign;    // flips the signs of two query elements where the scale is negative
    float scale_log2;       // |scale| * log2(e)
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
    size_t counters, joins, part, part_ml, bytes;   // offsets
};

constexpr AttnWorkspace attn_workspace(int head_dim, int rows) {
    const size_t slots = 2 * static_cast<size_t>(kAttnMaxCtas) * 16 * attn_row_warps(rows);
    AttnWorkspace w{};
    w.counters = kKvErrBytes;
    w.joins = w.counters + kAttnCounterBytes;
    w.part_ml = w.joins + kAttnMaxCtas * sizeof(int4);
    w.part = w.part_ml + slots * 2 * sizeof(float);
    w.bytes = w.part + slots * head_dim * sizeof(float);
    return w;
}

cudaError_t configure_attention();
cudaError_t launch_attention(int head_dim, const AttnParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_append(int head_dim, bool in_f32, const AppendParams& p, cudaStream_t stream);

}  // namespace qmmk
