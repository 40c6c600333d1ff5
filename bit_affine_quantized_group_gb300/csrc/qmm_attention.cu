// Attention of a step's new tokens over the paged cache.
//
// For one cache head the query rows (tokens x heads of the group) meet every
// visible position once: scores S = Q K^T and output O = P V are m16n8k16
// tensor-core products, and one pass over the cache keeps each row's running
// maximum m and sum l:
//   m' = max(m, S),  P = 2^(S - m'),  l = l 2^(m - m') + sum P,  O = O 2^(m - m') + P V.
// P enters the second product as two bfloat16 terms (P = hi + lo to 2^-17), so
// its rounding stays below that of the bfloat16 output.
//
// The bound is the cache's bytes: 4 D per position and cache head against
// 4 D rows operations. Every warp streams its own 16-position tiles through a
// ring of shared memory of its own with asynchronous copies, so the main loop
// has no block barrier and the copies of several tiles are always in flight.
//
// The positions of all (sequence, cache head, row group) items are laid end to
// end in units of 64 and cut into equal shares, one for each CTA of a grid that
// fills the GPU, by lengths read on the device: ragged lengths balance, and the
// launch does not depend on them. A head cut by a share's end leaves its parts
// (O, m, l) in the workspace; the CTA that arrives last joins them in order.
#include <cuda_bf16.h>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_kv.h"

namespace qmmk {

namespace {

template <int D>
struct AttnCfg {
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
    static constexpr int kSideBytes = kAttnTile * D * 2;          // the keys or the values of a tile
    static constexpr int kStageBytes = 2 * kSideBytes;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kSmem = kAttnWarps * kWarpBytes;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& d0, uint32_t& d1, uint32_t& d2,
                                                  uint32_t& d3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d0), "=r"(d1), "=r"(d2), "=r"(d3)
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// a and b as bfloat16 pairs: the rounded values and the rounded remainders.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}

__device__ __forceinline__ bool nonfinite_pair(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// The tiles of one sequence: those of the sinks, then from the window's first
// position to the end.
struct SeqSpan {
    int len;        // positions in the cache, at most what the page table holds
    int low;        // first position that the window shows to any row
    int sink_tiles;
    int low_tile;
    int tiles;

    __device__ __forceinline__ int units() const { return tiles == 0 ? 1 : (tiles + kAttnWarps - 1) / kAttnWarps; }
    __device__ __forceinline__ int tile_pos(int t) const {
        return (t < sink_tiles ? t : low_tile + t - sink_tiles) * kAttnTile;
    }
};

__device__ __forceinline__ SeqSpan span_of(const AttnParams& p, int seq) {
    SeqSpan s;
    const int most = p.max_pages << p.page_shift;
    int len = p.lengths[seq];
    if (len > most) {
        atomicOr(p.err, QMM_KV_BAD_LENGTH);
        len = most;
    }
    s.len = len > 0 ? len : 0;
    s.low = 0;
    s.low_tile = 0;
    s.sink_tiles = 0;
    if (p.window > 0) {
        const int64_t low = static_cast<int64_t>(s.len) - p.rows - p.window + 1;
        s.low = low > 0 ? static_cast<int>(low) : 0;
        s.low_tile = s.low / kAttnTile;
        const int64_t st = (static_cast<int64_t>(p.sinks) + kAttnTile - 1) / kAttnTile;
        s.sink_tiles = st < s.low_tile ? static_cast<int>(st) : s.low_tile;
    }
    s.tiles = s.sink_tiles + (s.len + kAttnTile - 1) / kAttnTile - s.low_tile;
    return s;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The first CTA whose share of `total` units reaches past unit u.
__device__ __forceinline__ int cta_of(int64_t u, int64_t total, int ctas) {
    return static_cast<int>(((u + 1) * ctas - 1) / total);
}

template <int D, int MT>
__global__ void __launch_bounds__(kAttnThreads, AttnCfg<D>::kCtasPerSm)
    qmm_attention_kernel(const __grid_constant__ AttnParams p) {
    using Cfg = AttnCfg<D>;
    constexpr int kRows = 16 * MT;
    constexpr int kChunks = D / 8;              // 16-byte chunks of a row
    constexpr int kRowsPerCopy = 32 / kChunks;  // rows that one copy instruction of a warp covers
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float s_ml[kAttnWarps][kRows][2];
    __shared__ uint32_t s_last;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane & 3, gid = lane >> 2;
    const uint32_t ring = smem_u32(smem) + warp * Cfg::kWarpBytes;

    griddep_launch_dependents();
    griddep_wait();

    // this CTA's share [u0, u1) of all units
    const int items = p.kv_heads * p.row_groups;
    int64_t total = 0;
    for (int s = lane; s < p.seqs; s += 32) total += span_of(p, s).units();
    total = warp_sum(total) * items;
    const int ctas = total < static_cast<int64_t>(gridDim.x) ? static_cast<int>(total) : static_cast<int>(gridDim.x);
    const int cta = blockIdx.x;
    if (cta >= ctas) return;
    int64_t u = total * cta / ctas;
    const int64_t u1 = total * (cta + 1) / ctas;

    // the sequence that unit u lies in, and the unit where it begins
    int seq = 0;
    int64_t base = 0;
    for (int s0 = 0; s0 < p.seqs; s0 += 32) {
        const int64_t mine = s0 + lane < p.seqs ? static_cast<int64_t>(span_of(p, s0 + lane).units()) * items : 0;
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, s0 + lane < p.seqs && base + upto > u);
        if (past != 0) {
            const int at = __ffs(past) - 1;
            seq = s0 + at;
            base += __shfl_sync(0xFFFFFFFFu, upto - mine, at);
            break;
        }
        base += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }

    while (u < u1) {
        const SeqSpan span = span_of(p, seq);
        const int units = span.units();
        const int64_t in_seq = u - base;
        if (in_seq >= static_cast<int64_t>(units) * items) {
            base += static_cast<int64_t>(units) * items;
            ++seq;
            continue;
        }
        const int item = static_cast<int>(in_seq / units);
        const int ua = static_cast<int>(in_seq - static_cast<int64_t>(item) * units);
        const int ub = static_cast<int>(u1 - u < units - ua ? ua + (u1 - u) : units);
        const int head = item / p.row_groups;
        const int row0 = (item - head * p.row_groups) * kRows;   // first query row of the group
        const int rows_left = p.rows * p.group - row0;
        const int rows = rows_left < kRows ? rows_left : kRows;
        const int first_pos = span.len - p.rows;                 // the position of the sequence's first new token

        const int t0 = ua * kAttnWarps + warp;
        const int t1 = ub * kAttnWarps < span.tiles ? ub * kAttnWarps : span.tiles;
        const int mine = t1 > t0 ? (t1 - t0 + kAttnWarps - 1) / kAttnWarps : 0;

        const uint16_t* kbase = p.k.base + head * p.k.head;
        const uint16_t* vbase = p.v.base + head * p.v.head;
        const int32_t* table = p.page_table + static_cast<int64_t>(seq) * p.max_pages;

        // lane l < 16 looks up the page of position l of a tile, one tile ahead of its copies
        auto page_of = [&](int i) -> int {
            if (i >= mine) return -1;
            const int pos = span.tile_pos(t0 + i * kAttnWarps) + (lane & 15);
            const bool seen = pos < span.len && (pos >= span.low || pos < p.sinks);
            return seen ? table[pos >> p.page_shift] : -1;
        };
        int next_page = page_of(0);
        auto issue = [&](int i) {
            if (i < mine) {
                const int pos = span.tile_pos(t0 + i * kAttnWarps) + (lane & 15);
                const bool seen = pos < span.len && (pos >= span.low || pos < p.sinks);
                const int page = next_page;
                const bool ok = seen && page >= 0 && page < p.num_pages;
                if (seen && !ok) atomicOr(p.err, QMM_KV_BAD_PAGE);
                const int slot = pos & ((1 << p.page_shift) - 1);
                const int64_t koff = ok ? page * p.k.page + slot * p.k.slot : 0;
                const int64_t voff = ok ? page * p.v.page + slot * p.v.slot : 0;
                const uint32_t valid = __ballot_sync(0xFFFFFFFFu, ok);
                next_page = page_of(i + 1);
                const uint32_t stage = ring + (i % Cfg::kStages) * Cfg::kStageBytes;
                const int chunk = lane % kChunks;
#pragma unroll
                for (int it = 0; it < kAttnTile / kRowsPerCopy; ++it) {
                    const int r = it * kRowsPerCopy + lane / kChunks;
                    const int64_t ko = __shfl_sync(0xFFFFFFFFu, koff, r);
                    const int64_t vo = __shfl_sync(0xFFFFFFFFu, voff, r);
                    const uint32_t bytes = (valid >> r) & 1u ? 16u : 0u;   // others are filled with zeros
                    const uint32_t dst = stage + r * (D * 2) + ((chunk ^ (r & 7)) << 4);
                    cp_async_16(dst, kbase + ko + chunk * 8, bytes);
                    cp_async_16(dst + Cfg::kSideBytes, vbase + vo + chunk * 8, bytes);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < Cfg::kStages - 1; ++i) issue(i);

        // query fragments: row = (token r, head g of the group)
        uint32_t qf[MT][D / 16][4];
        int row_pos[MT][2];   // the position of the lane's two rows of a tile; -1 for none
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = mt * 16 + h * 8 + gid;
                const bool in = i < rows;
                const int tok = (row0 + i) / p.group;
                const int g = row0 + i - tok * p.group;
                row_pos[mt][h] = in ? first_pos + tok : -1;
                const uint16_t* src = p.q + (static_cast<int64_t>(seq) * p.rows + (in ? tok : 0)) * p.q_stride +
                                      static_cast<int64_t>(head * p.group + (in ? g : 0)) * D + quad * 2;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    qf[mt][kk][h] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
                    qf[mt][kk][h + 2] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
                }
            }
        }

        float o[MT][D / 8][4];
        float m[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.0f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[mt][n][j] = 0.0f;
        }

        for (int i = 0; i < mine; ++i) {
            cp_async_wait<Cfg::kStages - 2>();
            __syncwarp();   // every lane's copies of tile i have landed, and tile i - 1 is used up
            issue(i + Cfg::kStages - 1);
            const uint32_t kst = ring + (i % Cfg::kStages) * Cfg::kStageBytes;
            const uint32_t vst = kst + Cfg::kSideBytes;
            const int pos0 = span.tile_pos(t0 + i * kAttnWarps);

            float sc[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[mt][n][j] = 0.0f;
            {
                const int r = (lane & 7) + ((lane >> 4) << 3);
                const uint32_t row = kst + r * (D * 2);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b0, b1, b2, b3;
                    ldmatrix_x4(row + (((kk * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4), b0, b1, b2, b3);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_bf16(sc[mt][0], qf[mt][kk], b0, b1);
                        mma_bf16(sc[mt][1], qf[mt][kk], b2, b3);
                    }
                }
            }

            // tiles that every row sees whole need no mask
            const bool all_past = pos0 + kAttnTile - 1 <= first_pos;
            const bool in_window = p.window == 0 || span.len - 1 - pos0 < p.window || pos0 + kAttnTile <= p.sinks;
            const bool whole = all_past && in_window;
            uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float alpha[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[4] = {sc[mt][0][2 * h] * p.scale_log2, sc[mt][0][2 * h + 1] * p.scale_log2,
                                  sc[mt][1][2 * h] * p.scale_log2, sc[mt][1][2 * h + 1] * p.scale_log2};
                    if (!whole) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int pos = pos0 + (j >> 1) * 8 + quad * 2 + (j & 1);
                            const int back = row_pos[mt][h] - pos;
                            if (back < 0 || (p.window != 0 && back >= p.window && pos >= p.sinks)) v[j] = -INFINITY;
                        }
                    }
                    float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    const float m_new = fmaxf(m[mt][h], top);
                    const float ref = m_new == -INFINITY ? 0.0f : m_new;
                    alpha[h] = m_new == m[mt][h] ? 1.0f : exp2_approx(m[mt][h] - ref);
                    m[mt][h] = m_new;
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j] = exp2_approx(v[j] - ref);
                        sum += v[j];
                    }
                    l[mt][h] = fmaf(l[mt][h], alpha[h], sum);
                    split_bf16(v[0], v[1], ph[mt][h], pl[mt][h]);
                    split_bf16(v[2], v[3], ph[mt][h + 2], pl[mt][h + 2]);
                }
                if (__any_sync(0xFFFFFFFFu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[mt][n][0] *= alpha[0];
                        o[mt][n][1] *= alpha[0];
                        o[mt][n][2] *= alpha[1];
                        o[mt][n][3] *= alpha[1];
                    }
                }
            }

            // A position that only some rows see weighs nothing in the others, but 0 * inf is not 0: where such a
            // tile holds a value that is not finite, each token's rows get a product of their own without what
            // they do not see.
            bool apart = false;
            if (!whole && p.rows > 1) {
                bool bad = false;
                for (int c = lane; c < Cfg::kSideBytes / 16; c += 32) {
                    const uint4 w = lds128(vst + c * 16);
                    bad |= nonfinite_pair(w.x) || nonfinite_pair(w.y) || nonfinite_pair(w.z) || nonfinite_pair(w.w);
                }
                apart = __any_sync(0xFFFFFFFFu, bad);
            }
            const int vr = (lane & 7) + (((lane >> 3) & 1) << 3);
            const uint32_t vrow = vst + vr * (D * 2);
            if (!apart) {
#pragma unroll
                for (int n = 0; n < D / 8; n += 2) {
                    uint32_t b0, b1, b2, b3;
                    ldmatrix_x4_trans(vrow + (((n + (lane >> 4)) ^ (vr & 7)) << 4), b0, b1, b2, b3);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_bf16(o[mt][n], ph[mt], b0, b1);
                        mma_bf16(o[mt][n + 1], ph[mt], b2, b3);
                        mma_bf16(o[mt][n], pl[mt], b0, b1);
                        mma_bf16(o[mt][n + 1], pl[mt], b2, b3);
                    }
                }
            } else {
                for (int r = 0; r < p.rows; ++r) {
                    const int rp = first_pos + r;
                    uint32_t keep[2];   // the halves of a fragment word whose position token r sees
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        keep[w] = 0u;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int pos = pos0 + w * 8 + quad * 2 + j;
                            const int back = rp - pos;
                            if (back >= 0 && (p.window == 0 || back < p.window || pos < p.sinks))
                                keep[w] |= 0xFFFFu << (16 * j);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < D / 8; n += 2) {
                        uint32_t b0, b1, b2, b3;
                        ldmatrix_x4_trans(vrow + (((n + (lane >> 4)) ^ (vr & 7)) << 4), b0, b1, b2, b3);
                        b0 &= keep[0], b2 &= keep[0], b1 &= keep[1], b3 &= keep[1];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            float x[4] = {}, y[4] = {};
                            mma_bf16(x, ph[mt], b0, b1);
                            mma_bf16(y, ph[mt], b2, b3);
                            mma_bf16(x, pl[mt], b0, b1);
                            mma_bf16(y, pl[mt], b2, b3);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (row_pos[mt][j >> 1] == rp) {
                                    o[mt][n][j] += x[j];
                                    o[mt][n + 1][j] += y[j];
                                }
                            }
                        }
                    }
                }
            }
        }

        // join the warps through the ring's memory
        cp_async_wait<0>();
        __syncthreads();
        float* const s_o = reinterpret_cast<float*>(smem) + warp * kRows * D;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum = l[mt][h];
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                const int row = mt * 16 + h * 8 + gid;
                if (quad == 0) {
                    s_ml[warp][row][0] = m[mt][h];
                    s_ml[warp][row][1] = sum;
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2*>(s_o + row * D + n * 8 + quad * 2) =
                        make_float2(o[mt][n][2 * h], o[mt][n][2 * h + 1]);
            }
        }
        __syncthreads();

        const int64_t g0 = base + static_cast<int64_t>(item) * units;   // the item's units [g0, g0 + units)
        const bool cut = ua != 0 || ub != units;
        const int slot = 2 * cta + (ua == 0 ? 1 : 0);
        auto out_row = [&](int i) -> uint16_t* {
            const int tok = (row0 + i) / p.group;
            const int g = row0 + i - tok * p.group;
            return p.out + (static_cast<int64_t>(seq) * p.rows + tok) * p.out_stride +
                   static_cast<int64_t>(head * p.group + g) * D;
        };
        for (int e = threadIdx.x; e < rows * (D / 4); e += kAttnThreads) {
            const int row = e / (D / 4), d = (e - row * (D / 4)) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_ml[w][row][0]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float a = exp2_approx(s_ml[w][row][0] - ref);
                sum = fmaf(s_ml[w][row][1], a, sum);
                const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                                  (w * kRows + row) * D + d);
                acc.x = fmaf(v.x, a, acc.x);
                acc.y = fmaf(v.y, a, acc.y);
                acc.z = fmaf(v.z, a, acc.z);
                acc.w = fmaf(v.w, a, acc.w);
            }
            if (!cut) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                *reinterpret_cast<uint2*>(out_row(row) + d) =
                    make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            } else {
                *reinterpret_cast<float4*>(p.part + (static_cast<int64_t>(slot) * kRows + row) * D + d) = acc;
                if (d == 0)
                    *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(slot) * kRows + row) * 2) =
                        make_float2(top, sum);
            }
        }
        if (cut) {
            const int c0 = cta_of(g0, total, ctas), c1 = cta_of(g0 + units - 1, total, ctas);
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) s_last = atomicAdd(p.counters + c0, 1u) == static_cast<uint32_t>(c1 - c0) ? 1u : 0u;
            __syncthreads();
            if (s_last != 0) {
                __threadfence();
                if (threadIdx.x == 0) p.counters[c0] = 0u;
                // the part of CTA c: its last item's slot where the item begins in it, else its first item's
                auto part_of = [&](int c, int row) -> int64_t {
                    return (static_cast<int64_t>(2 * c + (c == c0 ? 1 : 0))) * kRows + row;
                };
                for (int e = threadIdx.x; e < rows * (D / 4); e += kAttnThreads) {
                    const int row = e / (D / 4), d = (e - row * (D / 4)) * 4;
                    float top = -INFINITY;
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(p.part_ml + part_of(c, row) * 2));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    float sum = 0.0f;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) {
                        const int64_t at = part_of(c, row);
                        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + at * 2));
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part + at * D + d));
                        const float a = exp2_approx(ml.x - ref);
                        sum = fmaf(ml.y, a, sum);
                        acc.x = fmaf(v.x, a, acc.x);
                        acc.y = fmaf(v.y, a, acc.y);
                        acc.z = fmaf(v.z, a, acc.z);
                        acc.w = fmaf(v.w, a, acc.w);
                    }
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    *reinterpret_cast<uint2*>(out_row(row) + d) =
                        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                }
            }
        }
        __syncthreads();   // the ring is free for the next item's copies
        u += ub - ua;
    }
}

template <int D, int MT>
cudaError_t launch(const AttnParams& p0, int num_sms, cudaStream_t stream) {
    AttnParams p = p0;
    p.row_groups = (p.rows * p.group + 16 * MT - 1) / (16 * MT);
    int ctas = AttnCfg<D>::kCtasPerSm * num_sms;
    if (ctas > kAttnMaxCtas) ctas = kAttnMaxCtas;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = AttnCfg<D>::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qmm_attention_kernel<D, MT>, p);
}

template <int D, int MT>
cudaError_t configure() {
    return cudaFuncSetAttribute(qmm_attention_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnCfg<D>::kSmem);
}

}  // namespace

cudaError_t configure_attention() {
    cudaError_t e = configure<64, 1>();
    if (e == cudaSuccess) e = configure<64, 2>();
    if (e == cudaSuccess) e = configure<128, 1>();
    if (e == cudaSuccess) e = configure<128, 2>();
    if (e == cudaSuccess) e = configure<256, 1>();
    return e;
}

cudaError_t launch_attention(int head_dim, const AttnParams& p, int num_sms, cudaStream_t stream) {
    const bool two = attn_row_tiles(head_dim, p.rows * p.group) == 2;
    if (head_dim == 64) return two ? launch<64, 2>(p, num_sms, stream) : launch<64, 1>(p, num_sms, stream);
    if (head_dim == 128) return two ? launch<128, 2>(p, num_sms, stream) : launch<128, 1>(p, num_sms, stream);
    return launch<256, 1>(p, num_sms, stream);
}

}  // namespace qmmk
