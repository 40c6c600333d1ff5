// What the attention kernels over a paged cache share: the walk over the work, the copying warps, and the joining of parts.
// A configuration Cfg names the sizes: head_dim D, the bits of a cache's elements kBits (16: bfloat16, 8 or 4: codes), the
// query rows of a CTA kRows, its computing warps, and the room of its rings.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_kv.h"

namespace qmmk {

namespace {

constexpr int kStep = 64;       // positions of a step
constexpr int kJoin = 40;       // parts of a head that one CTA joins at once
constexpr int kJoinRun = 16;    // more of them: runs of this many first
constexpr int kJoinWarps = 8;   // of a CTA of the join kernel

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool copy) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16u : 0u) : "memory");
}

__device__ __forceinline__ void cp_async_pairs(uint32_t dst, const void* src, int bytes, bool copy) {
    const uint32_t n = copy ? bytes : 0;
    if (bytes == 16) asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
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

// A bounded wait on a phase, as mbar_wait, but inline (a call would keep the kernel from splitting its registers) and
// without the clock for the first tries: reading it took longer than most waits.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t code) {
    unsigned long long t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 1023u) == 0) {
            if (*reinterpret_cast<volatile uint32_t*>(err) & QMM_KV_TIMEOUT) return false;
            const unsigned long long now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) {
                atomicOr(err, code);
                return false;
            }
        }
    }
}

// The steps of one sequence: those of the sinks, then from the window's first position to the end.
struct SeqSpan {
    int len;        // positions in the cache, at most what the page table holds
    int first;      // position of the first new token, by the length as it is given
    int low;        // first position that the window shows to any row
    int sink_steps;
    int low_step;
    int steps;

    // in units of `unit` steps; a sequence without any has one, which writes its zeros
    __device__ __forceinline__ int units(int unit) const {
        if (unit == 1) return steps == 0 ? 1 : steps;
        return steps == 0 ? 1 : static_cast<uint32_t>(steps + unit - 1) / static_cast<uint32_t>(unit);
    }
    __device__ __forceinline__ int step_pos(int t) const {
        return (t < sink_steps ? t : low_step + t - sink_steps) * kStep;
    }
};

// `len`: of the sequence, 0 at least. Rows stand where it says even if it is more than the page table holds, as the append
// puts them.
__device__ __forceinline__ SeqSpan span_of(const AttnParams& p, int len) {
    SeqSpan s;
    s.len = min(len, p.positions);
    s.first = len - p.rows;
    s.low = 0;
    s.low_step = 0;
    s.sink_steps = 0;
    if (p.window > 0) {
        s.low = min(max(max(s.first, 0) - p.window + 1, 0), s.len);
        s.low_step = s.low / kStep;
        s.sink_steps = min((p.sinks + kStep - 1) / kStep, s.low_step);
    }
    s.steps = s.sink_steps + (s.len + kStep - 1) / kStep - s.low_step;
    return s;
}

__device__ __forceinline__ int length_of(const AttnParams& p, int seq) {
    if (seq >= p.seqs) return 0;
    const int len = p.lengths[seq];
    if (len > p.positions) atomicOr(p.err, QMM_KV_BAD_LENGTH);
    return len > 0 ? len : 0;
}

// Floor of a * b / c; a 64-bit division takes as long as a load.
__device__ __forceinline__ int mul_div(int a, int b, int c) {
    if (a < (1 << 22) && b <= 512) return static_cast<uint32_t>(a * b) / static_cast<uint32_t>(c);
    return static_cast<int>(static_cast<int64_t>(a) * b / c);
}

// The first CTA whose share of `total` units reaches past unit u.
__device__ __forceinline__ int cta_of(int u, int total, int ctas) {
    if (total < (1 << 22) && ctas <= 512) return (static_cast<uint32_t>((u + 1) * ctas) - 1) / static_cast<uint32_t>(total);
    return static_cast<int>((static_cast<int64_t>(u + 1) * ctas - 1) / total);
}

// A CTA's share of the units, item by item. Every warp walks it for itself; lane l holds the length of the sequence
// 32 b + l of the current block b. All units together are less than 2^31 (p.min_unit sees to that).
struct Share {
    int u, u1, total;
    int base;       // the unit that sequence `seq` begins at
    int ctas, unit, items, seq, lane_len;

    // Whole warps. False: nothing for this CTA.
    __device__ __forceinline__ bool init(const AttnParams& p, int short_share, int lane) {
        const int most = gridDim.x;
        items = p.kv_heads * p.row_groups;
        lane_len = length_of(p, lane);
        // Units of one step (p.min_unit steps). Where items are few, units of so many more that every CTA has one unit at
        // most, for a second item costs a CTA several steps: n of them if that makes the longest share at most 2/5 longer.
        // Shares of fewer steps than short_share are not worth the joining of more parts, nor two such shares that of two.
        int n = 1, low = 0, high = 0;   // units of `low` are too many
#pragma unroll 1
        for (;;) {
            int sum = 0, longest = 0;
#pragma unroll 1
            for (int s = lane; s < p.seqs; s += 32) {
                const SeqSpan span = span_of(p, s < 32 ? lane_len : length_of(p, s));
                sum += span.units(n * p.min_unit);
                longest = max(longest, span.steps);
            }
            sum = __reduce_add_sync(0xFFFFFFFFu, sum) * items;
            const bool first = high == 0;
            if (first || sum <= most) {
                high = n;
                unit = n * p.min_unit;
                total = sum;
            } else {
                low = n;
            }
            if (first) {
                if (p.seqs * items > most) break;
                n = static_cast<uint32_t>(sum + most - 1) / static_cast<uint32_t>(most);
                if (n < short_share)
                    n = __reduce_max_sync(0xFFFFFFFFu, longest) <= 2 * short_share ? 2 * short_share : short_share;
                low = n - 1;
                high = n * 7 / 5 + 1;
            } else {
                if (high - low <= 1) break;
                n = (low + high) / 2;
            }
        }
        ctas = total < static_cast<int>(gridDim.x) ? total : static_cast<int>(gridDim.x);
        const int cta = blockIdx.x;
        if (cta >= ctas) return false;
        u = ctas == total ? cta : mul_div(total, cta, ctas);
        u1 = ctas == total ? cta + 1 : mul_div(total, cta + 1, ctas);
        seq = 0;
        base = 0;
        if (p.seqs == 1) return true;
        for (int s0 = 0; s0 < p.seqs; s0 += 32) {
            if (s0 > 0) lane_len = length_of(p, s0 + lane);
            const int mine = s0 + lane < p.seqs ? span_of(p, lane_len).units(unit) * items : 0;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
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
        return true;
    }
};

struct Item {
    SeqSpan span;
    int g0;              // its first unit
    int seq, head, row0; // row0: its first query row of the group
    int units, ua, ub;   // units, and those [ua, ub) of this share
    int t0, steps;       // the first step of this share, and how many

    __device__ __forceinline__ bool next(const AttnParams& p, Share& s, int rows, int lane) {
        for (;;) {
            if (s.u >= s.u1) return false;
            seq = s.seq;
            span = span_of(p, __shfl_sync(0xFFFFFFFFu, s.lane_len, seq & 31));
            units = span.units(s.unit);
            if (s.u - s.base < units * s.items) break;
            s.base += units * s.items;
            if ((++s.seq & 31) == 0) s.lane_len = length_of(p, s.seq + lane);
        }
        const int item = units == 1 ? s.u - s.base : static_cast<uint32_t>(s.u - s.base) / static_cast<uint32_t>(units);
        g0 = s.base + item * units;
        ua = s.u - g0;
        ub = s.u1 - s.u < units - ua ? ua + (s.u1 - s.u) : units;
        head = p.row_groups == 1 ? item : item / p.row_groups;
        row0 = (item - head * p.row_groups) * rows;
        t0 = ua * s.unit;
        const int t1 = ub * s.unit < span.steps ? ub * s.unit : span.steps;
        steps = t1 > t0 ? t1 - t0 : 0;
        s.u += ub - ua;
        return true;
    }
};

// The parts of one cut head that CTAs c0, c0 + 1, ... leave: the CTA that it begins in stores its last item there, the
// others their first.
struct Parts {
    float* o;       // [slot][rows][D]
    float* ml;      // [slot][rows][2]
    int rows, c0;
    __device__ __forceinline__ int64_t row(int i, int r) const {
        return static_cast<int64_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)) * rows + r;
    }
};

// Join parts first, first + step, ... (n of them, at most kJoin) of `rows` query rows in that order; store(row, d,
// values, m, l) takes the sums. `weights` is shared memory for (n + 2) * rows floats, `room` for `room_bytes` of parts:
// loads to registers were six at a time and took 5 us for the 38 parts of 4 rows of 131,072 positions. The four copying
// warps do it.
template <int D, class Store>
__device__ __forceinline__ void join_parts(const Parts& parts, int first, int step, int n, int rows, float* weights,
                                           const float* room, int room_bytes, int tid, Store store) {
    const int warp = tid >> 5, lane = tid & 31;
    float* const sums = weights + n * rows;
    const int most = room_bytes / (n * D * 4);   // rows that have room at once
    const int together = rows < most ? rows : most;
    auto fetch = [&](int r0, int count) {
        for (int i = warp; i < n; i += 4) {
            const float* src = parts.o + parts.row(first + i * step, r0) * D;
            const uint32_t dst = smem_u32(room) + i * count * (D * 4);
            for (int e = lane; e < count * (D / 4); e += 32) cp_async_16(dst + e * 16, src + e * 4);
        }
    };
    fetch(0, together);
    for (int r = warp; r < rows; r += 4) {
        constexpr int kSets = (kJoin + 31) / 32;
        float2 ml[kSets];
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            const int i = k * 32 + lane;
            ml[k] = make_float2(-INFINITY, 0.0f);
            if (i < n) ml[k] = __ldcg(reinterpret_cast<const float2*>(parts.ml + parts.row(first + i * step, r) * 2));
        }
#pragma unroll
        for (int k = 0; k < kSets; ++k) top = fmaxf(top, ml[k].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float ref = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            const int i = k * 32 + lane;
            const float a = exp2_approx(ml[k].x - ref);
            if (i < n) weights[i * rows + r] = a;
            sum = fmaf(ml[k].y, a, sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) {
            sums[2 * r] = top;
            sums[2 * r + 1] = sum;
        }
    }
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += together) {
        const int count = rows - r0 < together ? rows - r0 : together;
        if (r0 > 0) {
            named_barrier(3, 128);
            fetch(r0, count);
        }
        cp_async_wait_all();
        named_barrier(3, 128);
        for (int e = tid; e < count * (D / 4); e += 128) {
            const int r = r0 + e / (D / 4), d = e % (D / 4) * 4;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(room + (i * count * (D / 4) + e) * 4);
                const float a = weights[i * rows + r];
                acc.x = fmaf(v.x, a, acc.x);
                acc.y = fmaf(v.y, a, acc.y);
                acc.z = fmaf(v.z, a, acc.z);
                acc.w = fmaf(v.w, a, acc.w);
            }
            store(r, d, acc, sums[2 * r], sums[2 * r + 1]);
        }
    }
}

// A head that a share cuts: its parts, the CTA that it begins in, and where it lies.
struct Cut {
    int n, c0, seq, head, row0, rows;
};

// The end of a cut head of up to 16 rows, by the four copying warps: the CTA that arrives last joins the parts, kJoin of
// them at once, more first in runs of kJoinRun.
template <class Cfg>
__device__ __forceinline__ void join_cut(const AttnParams& p, const Cut& cut, float* weights, const float* room,
                                         uint32_t* s_last, int tid) {
    constexpr int D = Cfg::kD;
    constexpr int kRoom = Cfg::kTeams * Cfg::kRingBytes;
    static_assert(kRoom >= kJoin * D * 4, "room for a row of every part");
    const int cta = blockIdx.x;
    const Parts parts{p.part, p.part_ml, Cfg::kRows, cut.c0};
    auto arrive = [&](uint32_t* counter, int of) -> bool {
        named_barrier(3, 128);   // every thread's stores come before the arrival
        if (tid == 0) {
            __threadfence();
            const bool last = atomicAdd(counter, 1u) == static_cast<uint32_t>(of - 1);
            if (last) *counter = 0u;   // for the next call
            __threadfence();
            *s_last = last ? 1u : 0u;
        }
        named_barrier(3, 128);
        return *s_last != 0;
    };
    const bool runs = cut.n > kJoin;
    if (runs) {
        const int run = (cta - cut.c0) / kJoinRun * kJoinRun;
        const int size = cut.n - run < kJoinRun ? cut.n - run : kJoinRun;
        // a last run of one part has nothing to wait for, and the next head may begin in its CTA and count there
        if (size > 1) {
            if (!arrive(p.counters + kAttnMaxCtas + cut.c0 + run, size)) return;
            join_parts<D>(parts, run, 1, size, cut.rows, weights, room, kRoom, tid,
                          [&](int r, int d, const float4& acc, float top, float sum) {
                              const int64_t at = parts.row(run, r);
                              *reinterpret_cast<float4*>(p.part + at * D + d) = acc;
                              if (d == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(top, sum);
                          });
        }
    }
    const int left = runs ? (cut.n + kJoinRun - 1) / kJoinRun : cut.n;
    if (!arrive(p.counters + cut.c0, left)) return;
    join_parts<D>(parts, 0, runs ? kJoinRun : 1, left, cut.rows, weights, room, kRoom, tid,
                  [&](int r, int d, const float4& acc, float, float sum) {
                      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                      const int row = cut.row0 + r, tok = (row * p.group_inverse) >> 20;
                      uint16_t* const dst = p.out + (static_cast<int64_t>(cut.seq) * p.rows + tok) * p.out_stride +
                                            static_cast<int64_t>(cut.head * p.group + row - tok * p.group) * D + d;
                      *reinterpret_cast<uint2*>(dst) =
                          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                  });
}

// The copying warps: keys and values of every step of the share into the ring, 16 positions of each side by each of the
// four. Shared-memory layout of a side: for each 64 elements of the heads 64 rows (positions) of 128 bytes, their
// 16-byte chunks c at place c ^ (row % 8). What no row sees, and what lies on a page outside the pool, is filled with
// zeros. (Tensor copies of the same boxes came to 35 GB/s for one CTA; these to over 80.)
template <class Cfg>
__device__ __forceinline__ void copy_share(const AttnParams& p, Share share, uint32_t rings, uint64_t* full,
                                           uint64_t* empty, float* weights, const float* room, uint32_t* s_last, int warp,
                                           int lane) {
    constexpr int kChunks = Cfg::kD / 8;              // 16-byte chunks of a row
    constexpr int kRowsPerCopy = 32 / kChunks;  // rows that one copy instruction of a warp covers
    constexpr int kCopies = 16 / kRowsPerCopy;
    constexpr int kPeriod = 8 / kRowsPerCopy;   // copies after which the places of chunks repeat
    const bool whole_pages = p.page_shift >= 4; // of 16 positions at least
    const int slot_mask = (1 << p.page_shift) - 1;
    const int chunk = lane % kChunks, r0 = lane / kChunks;
    uint32_t place[kPeriod];                    // of this lane's chunk in its ring side, by copy
#pragma unroll
    for (int k = 0; k < kPeriod; ++k) {
        const int r = k * kRowsPerCopy + r0;
        place[k] = rings + (chunk >> 3) * (kStep * 128) + (16 * warp + r) * 128 + (((chunk & 7) ^ (r & 7)) << 4);
    }
    int slot[Cfg::kTeams] = {}, round[Cfg::kTeams] = {};   // the next side of each team's ring
    bool alive = true;
    Cut first{}, last{};   // a share cuts at most its first and its last item
    Item it;
    while (it.next(p, share, Cfg::kRows, lane)) {
        if (Cfg::kInlineJoin && (it.ua != 0 || it.ub != it.units)) {
            const int c0 = cta_of(it.g0, share.total, share.ctas), left = p.rows * p.group - it.row0;
            const Cut cut{cta_of(it.g0 + it.units - 1, share.total, share.ctas) - c0 + 1, c0, it.seq, it.head, it.row0,
                          left < Cfg::kRows ? left : Cfg::kRows};
            if (first.n == 0) first = cut;
            else last = cut;
        }
        const SeqSpan span = it.span;
        const int32_t* table = p.page_table + static_cast<int64_t>(it.seq) * p.max_pages;
        const uint16_t* const bases[2] = {p.k.base + it.head * p.k.head + chunk * 8, p.v.base + it.head * p.v.head + chunk * 8};
        auto is_seen = [&](int pos) -> bool { return pos < span.len && (pos >= span.low || pos < p.sinks); };
        auto page_at = [&](int pos) -> int {
            const int page = table[pos >> p.page_shift];
            if (page >= 0 && page < p.num_pages) return page;
            atomicOr(p.err, QMM_KV_BAD_PAGE);
            return -1;
        };
        // Lane l knows the page of this warp's positions of the step i + l, -1 for none; those of the 32 steps after
        // are on their way.
        auto pages_of = [&](int i) -> int {
            if (!whole_pages || i + lane >= it.steps) return -1;
            const int pos = span.step_pos(it.t0 + i + lane) + 16 * warp;
            const int from = pos >= span.low || pos < p.sinks ? pos : span.low;   // the first that may be seen
            return from < span.len && from < pos + 16 ? page_at(from) : -1;
        };
        int pages = -1, next_pages = pages_of(0);
        auto copy_step = [&](int i, int team, int& slot, int& round) {
            if ((i & 31) == 0) {
                pages = next_pages;
                next_pages = pages_of(i + 32);
            }
            const int page = __shfl_sync(0xFFFFFFFFu, pages, i & 31);
            const int pos0 = span.step_pos(it.t0 + i) + 16 * warp;
            const bool all = page >= 0 && pos0 + 16 <= span.len && (pos0 >= span.low || pos0 + 16 <= p.sinks);
            const int slot0 = (pos0 & slot_mask) + r0;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int ring_slot = team * Cfg::kSides + slot;
                // a full round later the slot has been used and must have been read
                if (round > 0 && alive) alive = wait_phase(&empty[ring_slot], (round - 1) & 1, p.err, kErrEmptyWait);
                if (!alive) return;
                const KvSide& side = s == 0 ? p.k : p.v;
                const uint32_t dst = ring_slot * Cfg::kSideBytes;
                const uint16_t* src = bases[s] + (page < 0 ? 0 : page) * side.page + slot0 * side.slot;
                const int64_t step = kRowsPerCopy * side.slot;
                if (all) {
#pragma unroll
                    for (int k = 0; k < kCopies; ++k) {
                        cp_async_16(dst + place[k % kPeriod] + (k / kPeriod) * (8 * 128), src);
                        src += step;
                    }
                } else {
#pragma unroll 1
                    for (int k = 0; k < kCopies; ++k) {
                        const int r = k * kRowsPerCopy + r0, pos = pos0 + r;
                        int pg = is_seen(pos) ? page : -1;
                        if (!whole_pages && is_seen(pos)) {
                            pg = page_at(pos);
                            src = bases[s] + (pg < 0 ? 0 : pg) * side.page + (pos & slot_mask) * side.slot;
                        }
                        cp_async_16_or_zero(dst + place[0] + (r - r0) * 128 + ((((chunk ^ r) & 7) - ((chunk ^ r0) & 7)) << 4),
                                            pg < 0 ? bases[s] : src, pg >= 0);
                        src += step;
                    }
                }
                cp_async_arrive_noinc(&full[ring_slot]);
                if (++slot == Cfg::kSides) {
                    slot = 0;
                    ++round;
                }
            }
        };
        for (int i = 0; i < it.steps; i += Cfg::kTeams) {
#pragma unroll
            for (int team = 0; team < Cfg::kTeams; ++team)
                if (i + team < it.steps) copy_step(i + team, team, slot[team], round[team]);
        }
    }
    cp_async_wait_all();   // no copy lands after the CTA has ended, not even where the computing warps gave up waiting
    if constexpr (Cfg::kInlineJoin) {
        named_barrier(2, Cfg::kThreads);   // this share's parts are written, and its rings read
        if (first.n > 0) join_cut<Cfg>(p, first, weights, room, s_last, warp * 32 + lane);
        if (last.n > 0) join_cut<Cfg>(p, last, weights, room, s_last, warp * 32 + lane);
    }
}

// The copying warps of a cache of codes: the codes, scales and biases of keys and values of every step into a slot of the
// ring, 16 positions by each of the four. A slot has the keys' codes and pairs, then the values'; the configuration says
// where in a tile of 16 positions a chunk of 16 bytes lies. What a step costs a warp in instructions bounds short rows, so
// that 32 steps' addresses are computed at once, one by each lane, and passed on.
template <class Cfg>
__device__ __forceinline__ void copy_codes(const AttnParams& p, Share share, uint32_t rings, uint64_t* full, uint64_t* empty,
                                           float* weights, const float* room, uint32_t* s_last, int warp, int lane) {
    constexpr int kChunks = Cfg::kRowBytes / 16;   // 16-byte chunks of a row
    constexpr int kRowsPerCopy = 32 / kChunks;     // rows that one copy instruction of a warp covers
    constexpr int kCopies = 16 / kRowsPerCopy;
    constexpr int kPeriod = kRowsPerCopy < 8 ? 8 / kRowsPerCopy : 1;   // copies after which the places of chunks repeat
    constexpr int kPairsAt = kStep * Cfg::kRowBytes;   // of a side
    const bool whole_pages = p.page_shift >= 4;    // of 16 positions at least
    const int slot_mask = (1 << p.page_shift) - 1;
    const int chunk = lane % kChunks, r0 = lane / kChunks;
    uint32_t place[2][kPeriod];                    // of this lane's chunk of keys and of values in its ring slot, by copy
#pragma unroll
    for (int k = 0; k < kPeriod; ++k) {
        const int r = k * kRowsPerCopy + r0;
        place[0][k] = rings + 16 * warp * Cfg::kRowBytes + Cfg::key_place(r, chunk);
        place[1][k] = rings + Cfg::kSideBytes + 16 * warp * Cfg::kRowBytes + Cfg::value_place(r, chunk);
    }
    // lanes 0 to 15 copy the keys' pairs of a position each, the others the values'
    const int pair_row = lane & 15;
    const uint32_t pair_place = rings + (lane < 16 ? 0 : Cfg::kSideBytes) + kPairsAt + (16 * warp + pair_row) * Cfg::kPairBytes;
    const KvSide& pairs = lane < 16 ? p.ka : p.va;
    const int64_t step[2] = {kRowsPerCopy * p.k.slot, kRowsPerCopy * p.v.slot};
    int slot[Cfg::kTeams] = {}, round[Cfg::kTeams] = {};   // the next slot of each team's ring
    bool alive = true;
    Cut first{}, last{};   // a share cuts at most its first and its last item
    Item it;
    while (it.next(p, share, Cfg::kRows, lane)) {
        if (Cfg::kInlineJoin && (it.ua != 0 || it.ub != it.units)) {
            const int c0 = cta_of(it.g0, share.total, share.ctas), left = p.rows * p.group - it.row0;
            const Cut cut{cta_of(it.g0 + it.units - 1, share.total, share.ctas) - c0 + 1, c0, it.seq, it.head, it.row0,
                          left < Cfg::kRows ? left : Cfg::kRows};
            if (first.n == 0) first = cut;
            else last = cut;
        }
        const SeqSpan span = it.span;
        const int32_t* table = p.page_table + static_cast<int64_t>(it.seq) * p.max_pages;
        // of this lane's chunk in row r0 of a slice, and of its pair
        const uint8_t* const bases[2] = {
            reinterpret_cast<const uint8_t*>(p.k.base) + it.head * p.k.head + r0 * p.k.slot + chunk * 16,
            reinterpret_cast<const uint8_t*>(p.v.base) + it.head * p.v.head + r0 * p.v.slot + chunk * 16};
        const uint32_t* const pair_base = reinterpret_cast<const uint32_t*>(pairs.base) + it.head * pairs.head;
        auto is_seen = [&](int pos) -> bool { return pos < span.len && (pos >= span.low || pos < p.sinks); };
        auto page_at = [&](int pos) -> int {
            const int page = table[pos >> p.page_shift];
            if (page >= 0 && page < p.num_pages) return page;
            atomicOr(p.err, QMM_KV_BAD_PAGE);
            return -1;
        };
        // Lane l knows the page of this warp's positions of the step i + l, -1 for none; those of the 32 steps after
        // are on their way.
        auto pages_of = [&](int i) -> int {
            if (!whole_pages || i + lane >= it.steps) return -1;
            const int pos = span.step_pos(it.t0 + i + lane) + 16 * warp;
            const int from = pos >= span.low || pos < p.sinks ? pos : span.low;   // the first that may be seen
            return from < span.len && from < pos + 16 ? page_at(from) : -1;
        };
        int page = -1, next_page = pages_of(0);
        bool whole = false;              // this lane's step needs no look at single positions
        int64_t at[2] = {}, pair_at[2] = {};   // and lies there
        auto copy_step = [&](int i, int team, int& slot, int& round) {
            if ((i & 31) == 0) {
                page = next_page;
                next_page = pages_of(i + 32);
                const int pos = span.step_pos(it.t0 + i + lane) + 16 * warp;
                whole = page >= 0 && pos + 16 <= span.len && (pos >= span.low || pos + 16 <= p.sinks);
                const int64_t pg = page < 0 ? 0 : page, in = pos & slot_mask;
                at[0] = pg * p.k.page + in * p.k.slot;
                at[1] = pg * p.v.page + in * p.v.slot;
                pair_at[0] = pg * p.ka.page + in * p.ka.slot;
                pair_at[1] = pg * p.va.page + in * p.va.slot;
            }
            const int from = i & 31;
            const int ring_slot = team * Cfg::kSlots + slot;
            const bool all = __shfl_sync(0xFFFFFFFFu, whole, from);
            const int64_t src0 = __shfl_sync(0xFFFFFFFFu, at[0], from), src1 = __shfl_sync(0xFFFFFFFFu, at[1], from);
            const int64_t pair0 = __shfl_sync(0xFFFFFFFFu, pair_at[0], from), pair1 = __shfl_sync(0xFFFFFFFFu, pair_at[1], from);
            // a full round later the slot has been used and must have been read
            if (round > 0 && alive) alive = wait_phase(&empty[ring_slot], (round - 1) & 1, p.err, kErrEmptyWait);
            if (!alive) return;
            const uint32_t dst = ring_slot * Cfg::kSlotBytes;
            if (all) {
                const uint8_t* src[2] = {bases[0] + src0, bases[1] + src1};
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int k = 0; k < kCopies; ++k) {
                        cp_async_16(dst + place[s][k % kPeriod] + (k / kPeriod) * (8 * Cfg::kRowBytes), src[s]);
                        src[s] += step[s];
                    }
                cp_async_pairs(dst + pair_place, pair_base + (lane < 16 ? pair0 : pair1) + pair_row * pairs.slot, Cfg::kPairBytes, true);
            } else {
                const int pos0 = span.step_pos(it.t0 + i) + 16 * warp, own = __shfl_sync(0xFFFFFFFFu, page, from);
                auto page_of = [&](int pos) -> int { return !is_seen(pos) ? -1 : whole_pages ? own : page_at(pos); };
#pragma unroll 1
                for (int k = 0; k < kCopies; ++k) {
                    const int r = k * kRowsPerCopy + r0, pos = pos0 + r, pg = page_of(pos);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const KvSide& side = s == 0 ? p.k : p.v;
                        const uint8_t* from_row = bases[s];
                        if (pg >= 0) from_row += pg * side.page + ((pos & slot_mask) - r0) * side.slot;
                        const int to = s == 0 ? Cfg::key_place(r, chunk) : Cfg::kSideBytes + Cfg::value_place(r, chunk);
                        cp_async_16_or_zero(rings + dst + 16 * warp * Cfg::kRowBytes + to, from_row, pg >= 0);
                    }
                }
                const int pos = pos0 + pair_row, pg = page_of(pos);
                cp_async_pairs(dst + pair_place, pair_base + (pg < 0 ? 0 : pg * pairs.page + (pos & slot_mask) * pairs.slot),
                               Cfg::kPairBytes, pg >= 0);
            }
            cp_async_arrive_noinc(&full[ring_slot]);
            if (++slot == Cfg::kSlots) {
                slot = 0;
                ++round;
            }
        };
        for (int i = 0; i < it.steps; i += Cfg::kTeams) {
#pragma unroll
            for (int team = 0; team < Cfg::kTeams; ++team)
                if (i + team < it.steps) copy_step(i + team, team, slot[team], round[team]);
        }
    }
    cp_async_wait_all();   // no copy lands after the CTA has ended, not even where the computing warps gave up waiting
    if constexpr (Cfg::kInlineJoin) {
        named_barrier(2, Cfg::kThreads);   // this share's parts are written, and its rings read
        if (first.n > 0) join_cut<Cfg>(p, first, weights, room, s_last, warp * 32 + lane);
        if (last.n > 0) join_cut<Cfg>(p, last, weights, room, s_last, warp * 32 + lane);
    }
}

// Joins the parts of the cut heads, one row a warp.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) qmm_attention_join_kernel(const __grid_constant__ AttnParams p, int rows,
                                                                            int ctas) {
    __shared__ float s_weight[kJoinWarps][kAttnMaxCtas];
    __shared__ int s_list[kAttnMaxCtas];
    __shared__ int s_votes[2 * kJoinWarps];
    constexpr int kLanes = D / 4 < 32 ? D / 4 : 32;   // lanes of a row's output; the others take every second part
    constexpr int kSteps = D / 4 / kLanes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    // the CTAs that a cut head begins in
    static_assert(kAttnMaxCtas <= 64 * kJoinWarps, "two entries a thread");
    const int c_lo = threadIdx.x, c_hi = threadIdx.x + 32 * kJoinWarps;
    const bool has_lo = c_lo < ctas && p.joins[c_lo].x != 0, has_hi = c_hi < ctas && p.joins[c_hi].x != 0;
    const uint32_t votes_lo = __ballot_sync(0xFFFFFFFFu, has_lo), votes_hi = __ballot_sync(0xFFFFFFFFu, has_hi);
    if (lane == 0) s_votes[warp] = __popc(votes_lo), s_votes[kJoinWarps + warp] = __popc(votes_hi);
    __syncthreads();
    int before_lo = 0, before_hi = 0, count = 0;
#pragma unroll
    for (int w = 0; w < 2 * kJoinWarps; ++w) {
        if (w < warp) before_lo += s_votes[w];
        if (w < kJoinWarps + warp) before_hi += s_votes[w];
        count += s_votes[w];
    }
    if (has_lo) s_list[before_lo + __popc(votes_lo & ((1u << lane) - 1u))] = c_lo;
    if (has_hi) s_list[before_hi + __popc(votes_hi & ((1u << lane) - 1u))] = c_hi;
    __syncthreads();
    for (int task = blockIdx.x * kJoinWarps + warp; task < count * rows; task += gridDim.x * kJoinWarps) {
        const int c0 = s_list[task / rows], r = task % rows;
        const int4 join = p.joins[c0];
        const int n = join.x, seq = join.y, head = join.z, row0 = join.w;
        if (row0 + r >= p.rows * p.group) continue;
        const Parts parts{p.part, p.part_ml, rows, c0};
        float* const weight = s_weight[warp];
        __syncwarp();
        float top = -INFINITY, sum = 0.0f;
        if (n <= 32) {
            float2 ml = make_float2(-INFINITY, 0.0f);
            if (lane < n) ml = *reinterpret_cast<const float2*>(parts.ml + parts.row(lane, r) * 2);
            top = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float a = exp2_approx(ml.x - (top == -INFINITY ? 0.0f : top));
            weight[lane] = a;
            sum = ml.y * a;
        } else {
            for (int i = lane; i < n; i += 32) {
                const float m = parts.ml[parts.row(i, r) * 2];
                weight[i] = m;
                top = fmaxf(top, m);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float ref = top == -INFINITY ? 0.0f : top;
            for (int i = lane; i < n; i += 32) {
                const float a = exp2_approx(weight[i] - ref);
                weight[i] = a;
                sum = fmaf(parts.ml[parts.row(i, r) * 2 + 1], a, sum);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        __syncwarp();
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int tok = (row0 + r) / p.group;
        uint16_t* const dst = p.out + (static_cast<int64_t>(seq) * p.rows + tok) * p.out_stride +
                              static_cast<int64_t>(head * p.group + row0 + r - tok * p.group) * D;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int d = (k * kLanes + lane % kLanes) * 4;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            constexpr int kAtOnce = 12, kEvery = 32 / kLanes;   // loads in flight, also for the rest
            for (int i0 = lane / kLanes; i0 < n; i0 += kAtOnce * kEvery) {
                float4 v[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (i0 + i * kEvery < n)
                        v[i] = *reinterpret_cast<const float4*>(parts.o + parts.row(i0 + i * kEvery, r) * D + d);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    if (i0 + i * kEvery >= n) continue;
                    const float a = weight[i0 + i * kEvery];
                    acc.x = fmaf(v[i].x, a, acc.x);
                    acc.y = fmaf(v[i].y, a, acc.y);
                    acc.z = fmaf(v[i].z, a, acc.z);
                    acc.w = fmaf(v[i].w, a, acc.w);
                }
            }
#pragma unroll
            for (int o = kLanes; o < 32; o <<= 1) {
                acc.x += __shfl_xor_sync(0xFFFFFFFFu, acc.x, o);
                acc.y += __shfl_xor_sync(0xFFFFFFFFu, acc.y, o);
                acc.z += __shfl_xor_sync(0xFFFFFFFFu, acc.z, o);
                acc.w += __shfl_xor_sync(0xFFFFFFFFu, acc.w, o);
            }
            if (lane < kLanes)
                *reinterpret_cast<uint2*>(dst + d) =
                    make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        }
    }
}

template <class Cfg>
cudaError_t launch(void (*kernel)(AttnParams), const AttnParams& p0, int num_sms, cudaStream_t stream) {
    AttnParams p = p0;
    p.row_groups = (p.rows * p.group + Cfg::kRows - 1) / Cfg::kRows;
    // steps of the smallest unit: more than one only where all units might not fit 31 bits
    const int64_t steps = (static_cast<int64_t>(p.max_pages) << p.page_shift) / kStep + 2;
    p.min_unit = 1;
    while (steps / p.min_unit * p.seqs * p.kv_heads * p.row_groups >= (1LL << 30)) p.min_unit *= 2;
    int ctas = Cfg::kCtasPerSm * num_sms;
    if (ctas > kAttnMaxCtas) ctas = kAttnMaxCtas;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess || Cfg::kInlineJoin) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * num_sms));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, qmm_attention_join_kernel<Cfg::kD>, p, Cfg::kRows, ctas);
}

template <class Cfg>
cudaError_t configure(void (*kernel)(AttnParams)) {
    // a register split would wait forever for registers that the launch did not get
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e != cudaSuccess) return e;
    if (Cfg::kSplitRegs && a.numRegs < Cfg::kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
}

}  // namespace

}  // namespace qmmk
