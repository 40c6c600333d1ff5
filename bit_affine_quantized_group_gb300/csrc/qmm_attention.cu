// Attention of a step's new tokens over the paged cache.
//
// For one cache head the query rows (tokens x heads of the group) meet every
// visible position once: scores S = Q K^T and output O = P V are m16n8k16
// tensor-core products, and one pass over the cache keeps each row's running
// maximum m and sum l:
//   m' = max(m, S),  P = 2^(S - m'),  l = l 2^(m - m') + sum P,  O = O 2^(m - m') + P V.
// P enters the second product as two bfloat16 terms (P = hi + lo to 2^-16), so
// its rounding stays below that of the bfloat16 output.
//
// The bound is the cache's bytes: 4 D per position and cache head against
// 4 D rows operations. Four warps of a CTA do nothing but start asynchronous
// copies of the pages' rows into a ring of shared memory, keys and values of 64
// positions in turn, and run ahead over the ends of heads and sequences as far
// as the ring reaches; the others compute.
//
// The positions of all (sequence, cache head, row group) items are laid end to
// end in steps of 64 and cut into equal shares, one for each CTA of a grid that
// fills the GPU, by lengths read on the device: ragged lengths balance, and the
// launch does not depend on them. Few items are cut so that no share has parts
// of two. A head cut by a share's end leaves its parts (O, m, l) in the
// workspace. The CTA that arrives last joins them in order, or a second kernel
// does where there are more than 16 rows: one CTA would read them for too long.
//
// Measured with 8 cache heads of 128: 1 x 131,072 positions 88 us, 6.1 TB/s; 64
// ragged sequences 186 us, 6.0 TB/s; 1 x 257 positions 8.0 us, latency. With 4
// of them, 4 sequences x 8 tokens (64 rows) take 34 us, 14 of it products at
// mma.sync's rate; 24 sequences with a window of 4,096 and 2 heads of 256 take
// 48 us, 4.0 TB/s, a quarter of it start and join.
#include <cuda_bf16.h>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_kv.h"

namespace qmmk {

namespace {

constexpr int kStep = 64;       // positions of a step
constexpr int kJoin = 40;       // parts of a head that one CTA joins at once
constexpr int kJoinRun = 16;    // more of them: runs of this many first
constexpr int kJoinWarps = 8;   // of a CTA of the join kernel

// The computing warps form teams that take the steps in turn. Each warp of a team has all the positions of the step for
// 16 of up to 64 query rows, or with fewer row tiles a part of the positions: 32 where it can, for a step's chain of
// products, maximum and exponentials takes little longer for 32 positions than for 16. The outputs of 16 rows take D / 2
// registers of every lane, so that an SM has room for 8 computing warps: two CTAs of four, or one of eight for 256-wide
// heads.
template <int D, int RW>
struct AttnCfg {
    static constexpr int kCompute = D == 256 ? 8 : 4;              // computing warps
    static constexpr int kTeamWarps = RW == 1 && D < 256 ? 2 : 4;
    static constexpr int kTeams = kCompute / kTeamWarps;
    static constexpr int kParts = kTeamWarps / RW;                 // parts of a step's positions
    static constexpr int kTiles = 4 / kParts;                      // 16-position tiles of a part
    static constexpr int kGroups = kTeams * kParts;                // sets of positions of a row
    static constexpr bool kScaled = kGroups == 8;                  // groups join outputs of a common scale
    static constexpr int kThreads = 32 * (kCompute + 4);           // and a group of four that starts the copies
    // registers a thread: at launch, and then of the computing and the copying group, out of the same sum
    static constexpr int kLaunchRegs = D == 256 ? 168 : 128;
    static constexpr int kComputeRegs = D == 256 ? 216 : 184;
    static constexpr int kCopyRegs = 72;
    static_assert(kCompute * kComputeRegs + 4 * kCopyRegs <= (kCompute + 4) * kLaunchRegs, "registers of a CTA");
    static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
    // steps of the shortest share: about as long as joining parts takes, and work for every team
    static constexpr int kShortShare = RW == 1 && D < 256 ? 4 : RW == 4 ? kTeams : 2;
    static constexpr int kSideBytes = kStep * D * 2;               // the keys or the values of a step
    // Every team has a ring of its own: in a common one, a team that only steps over the other's sides could take a
    // barrier's phase for one two rounds away.
    static constexpr int kSides = (D == 64 ? 12 : 6) / kTeams - (D > 64 && RW == 4 ? 1 : 0);
    static constexpr int kJoinCols = D == 256 ? 32 : 64;           // columns of all rows that the groups join at once
    static constexpr int kRingBytes = kSides * kSideBytes;         // of a team
    static constexpr int kJoinBytes = kGroups * 16 * RW * kJoinCols * 4;
    static constexpr bool kQueryRegs = D == 64 || (D == 128 && RW < 4);   // else the queries stay in shared memory
    static constexpr bool kAhead = D < 256 || RW < 4;              // fragments are read one product ahead
    static constexpr int kQueryBytes = 16 * D * 2;                 // of a row tile
    // shared memory: rings, join, queries, maxima and sums, barriers
    static constexpr int kJoinAt = kTeams * kRingBytes;
    static constexpr int kQueryAt = kJoinAt + kJoinBytes;
    static constexpr int kMlAt = kQueryAt + (kQueryRegs ? 0 : RW * kQueryBytes);
    static constexpr int kSumAt = kMlAt + kGroups * 16 * RW * 8;
    static constexpr int kBarsAt = kSumAt + (kScaled ? 16 * RW * 8 : 0);
    static constexpr int kLastAt = kBarsAt + 2 * kTeams * kSides * 8;
    static constexpr int kSmem = kLastAt + 16;
    static_assert((kJoin + 2) * 16 * 4 <= kJoinBytes, "the weights of a join fit its buffer");
    static_assert(kSmem <= (D == 256 ? 227 * 1024 : 113 * 1024), "shared memory of an SM");
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool copy) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16u : 0u) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& d0, uint32_t& d1, uint32_t& d2,
                                                  uint32_t& d3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d0), "=r"(d1), "=r"(d2), "=r"(d3)
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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

// Weights a and b, at least 0, as bfloat16 pairs: their upper halves, and the rounded remainders (hi + lo is within 2^-16).
// The remainders get 2^-24 of the upper halves more, so that no weight from 2^-109 on has a lo of 0: that times an infinite
// value were NaN where the weight times it is infinite. (Below, weights of no more than 8 bits still have one.)
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
    constexpr float kLess = 1.0f - 0x1p-24f;
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    hi = __byte_perm(ua, ub, 0x7632);
    lo = pack_bf16(fmaf(__uint_as_float(ua & 0xFFFF0000u), -kLess, a), fmaf(__uint_as_float(ub & 0xFFFF0000u), -kLess, b));
}

__device__ __forceinline__ bool nonfinite_pair(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
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
template <int D, int RW>
__device__ __forceinline__ void join_cut(const AttnParams& p, const Cut& cut, float* weights, const float* room,
                                         uint32_t* s_last, int tid) {
    constexpr int kRoom = AttnCfg<D, RW>::kTeams * AttnCfg<D, RW>::kRingBytes;
    static_assert(kRoom >= kJoin * D * 4, "room for a row of every part");
    const int cta = blockIdx.x;
    const Parts parts{p.part, p.part_ml, 16 * RW, cut.c0};
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
template <int D, int RW>
__device__ __forceinline__ void copy_share(const AttnParams& p, Share share, uint32_t rings, uint64_t* full,
                                           uint64_t* empty, float* weights, const float* room, uint32_t* s_last, int warp,
                                           int lane) {
    using Cfg = AttnCfg<D, RW>;
    constexpr int kChunks = D / 8;              // 16-byte chunks of a row
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
    while (it.next(p, share, 16 * RW, lane)) {
        if (RW == 1 && (it.ua != 0 || it.ub != it.units)) {
            const int c0 = cta_of(it.g0, share.total, share.ctas), left = p.rows * p.group - it.row0;
            const Cut cut{cta_of(it.g0 + it.units - 1, share.total, share.ctas) - c0 + 1, c0, it.seq, it.head, it.row0,
                          left < 16 * RW ? left : 16 * RW};
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
    if constexpr (RW == 1) {
        named_barrier(2, Cfg::kThreads);   // this share's parts are written, and its rings read
        if (first.n > 0) join_cut<D, RW>(p, first, weights, room, s_last, warp * 32 + lane);
        if (last.n > 0) join_cut<D, RW>(p, last, weights, room, s_last, warp * 32 + lane);
    }
}

template <int D, int RW>
__global__ void __launch_bounds__(AttnCfg<D, RW>::kThreads, AttnCfg<D, RW>::kCtasPerSm)
    qmm_attention_kernel(const __grid_constant__ AttnParams p) {
    using Cfg = AttnCfg<D, RW>;
    constexpr int kRows = 16 * RW;              // query rows of a CTA
    constexpr int kGroups = Cfg::kGroups;
    constexpr int kTiles = Cfg::kTiles;
    constexpr int kPartRows = 16 * kTiles;      // positions of a warp's part of a step
    constexpr int kThreads = 32 * Cfg::kCompute;   // computing threads
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* const full = reinterpret_cast<uint64_t*>(smem + Cfg::kBarsAt);
    uint64_t* const empty = full + Cfg::kTeams * Cfg::kSides;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(smem);
    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::kTeams * Cfg::kSides; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&empty[i], Cfg::kTeamWarps);
        }
        fence_barrier_init();
    }
    __syncthreads();
    griddep_launch_dependents();
    griddep_wait();

    Share share;
    const bool any = share.init(p, Cfg::kShortShare, lane);
    float* const s_join = reinterpret_cast<float*>(smem + Cfg::kJoinAt);
    uint32_t* const s_last = reinterpret_cast<uint32_t*>(smem + Cfg::kLastAt);
    if (RW > 1 && threadIdx.x == 0) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (!any) return;
    if (warp >= Cfg::kCompute) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kCopyRegs));
        copy_share<D, RW>(p, share, ring, full, empty, s_join, reinterpret_cast<const float*>(smem), s_last, warp - Cfg::kCompute,
                          lane);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kComputeRegs));

    const int team = warp / Cfg::kTeamWarps;    // takes the steps team, team + kTeams, ... of every item
    const int part = warp % Cfg::kTeamWarps / RW;   // its part of the step's positions
    const int wr = warp % RW;                   // its row tile
    const int grp = team * Cfg::kParts + part;
    const int quad = lane & 3, gid = lane >> 2;
    const uint32_t q_smem = ring + Cfg::kQueryAt + wr * Cfg::kQueryBytes;
    float* const s_ml = reinterpret_cast<float*>(smem + Cfg::kMlAt);     // [kGroups][kRows][2]
    float* const s_sum = reinterpret_cast<float*>(smem + Cfg::kSumAt);   // [kRows][2]

    // fragment addresses in a side: the row of the lane's part, and the places of its four chunks of 64 elements
    const int kr = (lane & 7) + ((lane >> 4) << 3), vr = (lane & 7) + (((lane >> 3) & 1) << 3);
    uint32_t k_at[4], v_at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        k_at[j] = part * (kPartRows * 128) + kr * 128 + (((2 * j + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
        v_at[j] = part * (kPartRows * 128) + vr * 128 + (((2 * j + (lane >> 4)) ^ (lane & 7)) << 4);
    }

    uint64_t* const my_full = full + team * Cfg::kSides;
    uint64_t* const my_empty = empty + team * Cfg::kSides;
    int slot = 0, round = 0;   // of the next side in the team's ring
    bool alive = true;
    auto side_full = [&]() -> uint32_t {
        if (alive) alive = wait_phase(&my_full[slot], round & 1, p.err, kErrFullWait);
        return ring + (team * Cfg::kSides + slot) * Cfg::kSideBytes;
    };
    auto side_done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&my_empty[slot]);
        if (++slot == Cfg::kSides) {
            slot = 0;
            ++round;
        }
    };

    Item it;
    while (it.next(p, share, kRows, lane)) {
        const SeqSpan span = it.span;
        const int seq = it.seq, head = it.head, row0 = it.row0;
        const int rows_left = p.rows * p.group - row0;
        const int rows = rows_left < kRows ? rows_left : kRows;
        const int first_pos = span.first;
        auto seq_end = [&]() -> int { return min(first_pos + p.rows, p.positions); };   // span.len again

        // query row = (token, head of the group)
        auto token_of = [&](int i) -> int { return ((row0 + i) * p.group_inverse) >> 20; };   // (row0 + i) / group
        auto row_offset = [&](int i, int64_t stride) -> int64_t {
            const int tok = token_of(i);
            return (static_cast<int64_t>(seq) * p.rows + tok) * stride +
                   static_cast<int64_t>(head * p.group + row0 + i - tok * p.group) * D;
        };
        uint32_t qf[Cfg::kQueryRegs ? D / 16 : 1][4];
        int row_pos[2];   // the positions of the lane's two rows; -1 for none
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = wr * 16 + h * 8 + gid;
            const bool in = i < rows;
            row_pos[h] = in ? first_pos + token_of(i) : -1;
            if constexpr (Cfg::kQueryRegs) {
                const uint16_t* src = p.q + (in ? row_offset(i, p.q_stride) : 0) + quad * 2;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    qf[kk][h] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16) ^ p.query_sign : 0u;
                    qf[kk][h + 2] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) ^ p.query_sign : 0u;
                }
            }
        }
        if constexpr (!Cfg::kQueryRegs) {
            // every group has the same rows: each of its warps brings a share of its row tile
            constexpr int kRowsPerLoad = 32 / (D / 8);
            constexpr int kLoads = 16 / kRowsPerLoad / kGroups > 0 ? 16 / kRowsPerLoad / kGroups : 1;
            uint4 v[kLoads];
            const int c = lane % (D / 8);
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int i = wr * 16 + (k * kGroups + grp) * kRowsPerLoad + lane / (D / 8);
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (i < rows) v[k] = *reinterpret_cast<const uint4*>(p.q + row_offset(i, p.q_stride) + c * 8);
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int r = (k * kGroups + grp) * kRowsPerLoad + lane / (D / 8);
                v[k].x ^= p.query_sign, v[k].y ^= p.query_sign, v[k].z ^= p.query_sign, v[k].w ^= p.query_sign;
                if (r < 16) sts128(q_smem + r * (D * 2) + ((c ^ (r & 7)) << 4), v[k]);
            }
            named_barrier(1, kThreads);
        }

        float o[D / 8][4];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][j] = 0.0f;

        for (int i = team; i < it.steps; i += Cfg::kTeams) {
            const int pos0 = span.step_pos(it.t0 + i) + part * kPartRows;   // the warp's first position
            const uint32_t kst = side_full();

            // A single tile's two products run as two chains each, of the even and the odd parts of the sum.
            constexpr int kChains = kTiles == 1 ? 2 : 1;
            float sc[kChains][2 * kTiles][4];
#pragma unroll
            for (int c = 0; c < kChains; ++c)
#pragma unroll
                for (int n = 0; n < 2 * kTiles; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[c][n][j] = 0.0f;
            auto load_keys = [&](int kk, uint32_t(&b)[kTiles][4]) {
#pragma unroll
                for (int s = 0; s < kTiles; ++s)
                    ldmatrix_x4(kst + k_at[kk & 3] + (kk >> 2) * (kStep * 128) + s * (16 * 128), b[s][0], b[s][1], b[s][2],
                                b[s][3]);
            };
            auto load_query = [&](int kk, uint32_t(&a)[4]) {
                if constexpr (Cfg::kQueryRegs) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j] = qf[kk][j];
                } else {
                    ldmatrix_x4(q_smem + (lane & 15) * (D * 2) + (((kk * 2 + (lane >> 4)) ^ (lane & 7)) << 4), a[0], a[1],
                                a[2], a[3]);
                }
            };
            // the fragments of the next products are read before the present ones
            constexpr int kAhead = Cfg::kAhead ? 1 : 0;
            uint32_t kb[kAhead + 1][kTiles][4], qa[kAhead + 1][4];
            if constexpr (kAhead) {
                load_keys(0, kb[0]);
                load_query(0, qa[0]);
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                if (kk + kAhead < D / 16) {
                    load_keys(kk + kAhead, kb[(kk + 1) & kAhead]);
                    load_query(kk + kAhead, qa[(kk + 1) & kAhead]);
                }
#pragma unroll
                for (int s = 0; s < kTiles; ++s) {
                    const uint32_t(&b)[4] = kb[kk & kAhead][s];
                    mma_bf16(sc[kk % kChains][2 * s], qa[kk & kAhead], b[0], b[1]);
                    mma_bf16(sc[kk % kChains][2 * s + 1], qa[kk & kAhead], b[2], b[3]);
                }
            }
            side_done();

            // positions that every row sees need no mask
            const bool whole = pos0 + 16 * kTiles <= min(first_pos + 1, p.positions) &&
                               (p.window == 0 || first_pos + p.rows - 1 - pos0 < p.window || pos0 + 16 * kTiles <= p.sinks);
            float alpha[2];
            float pr[kTiles][2][4];   // scores, then weights: [tile][row of the lane][position]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int s = 0; s < kTiles; ++s) {
                    float(&v)[4] = pr[s][h];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x = sc[0][2 * s + (j >> 1)][2 * h + (j & 1)];
                        if constexpr (kChains == 2) x += sc[1][2 * s + (j >> 1)][2 * h + (j & 1)];
                        v[j] = x;
                    }
                    if (!whole) {
                        // position s * 16 + (j >> 1) * 8 + (j & 1) of the lane's lies after its row or the table's end, or
                        // before the window and past the sinks
                        const int own = row_pos[h] - pos0 - quad * 2;
                        const int last = min(own, seq_end() - 1 - pos0 - quad * 2);
                        // (in 32 bits without a sign: wraps for rows without a position, which see nothing anyway)
                        const int out = p.window == 0 ? -1 : static_cast<int>(static_cast<uint32_t>(own) - p.window);
                        const int sink = p.window == 0 ? -1 : p.sinks - pos0 - quad * 2;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int at = s * 16 + (j >> 1) * 8 + (j & 1);
                            if (at > last || (at <= out && at >= sink)) v[j] = -INFINITY;
                        }
                    }
                    top = fmaxf(top, fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
                }
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // scale_log2 is not negative (the queries take its sign), so that it keeps the order
                const float m_new = fmaxf(m[h], top == -INFINITY ? top : top * p.scale_log2);
                const float ref = m_new == -INFINITY ? 0.0f : m_new;
                alpha[h] = m_new == m[h] ? 1.0f : exp2_approx(m[h] - ref);
                m[h] = m_new;
                float sum = 0.0f;
#pragma unroll
                for (int s = 0; s < kTiles; ++s) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        pr[s][h][j] = exp2_approx(fmaf(pr[s][h][j], p.scale_log2, -ref));
                        sum += pr[s][h][j];
                    }
                }
                l[h] = fmaf(l[h], alpha[h], sum);
            }
            if (__any_sync(0xFFFFFFFFu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= alpha[0];
                    o[n][1] *= alpha[0];
                    o[n][2] *= alpha[1];
                    o[n][3] *= alpha[1];
                }
            }

            const uint32_t vst = side_full();
            // A position that only some rows see weighs nothing in the others, but 0 * inf is not 0: where such a
            // part of a step holds a value that is not finite, each token's rows get a product of their own without
            // what they do not see.
            bool apart = false;
            if (!whole && p.rows > 1) {
                bool bad = false;
                auto look = [&](int first, int end) {   // positions [first, end) of the part; they may be far from it
                    first = min(max(first, 0), kPartRows);
                    end = min(max(end, 0), kPartRows);
                    for (int c = first * (D / 8) + lane; c < end * (D / 8); c += 32) {
                        const uint32_t at = (part * kPartRows + c / (D / 8)) * 128 + ((c % (D / 8)) >> 3) * (kStep * 128);
                        const uint4 w = lds128(vst + at + ((c & 7) << 4));
                        bad |= nonfinite_pair(w.x) || nonfinite_pair(w.y) || nonfinite_pair(w.z) || nonfinite_pair(w.w);
                    }
                };
                look(first_pos + 1 - pos0, seq_end() - pos0);                                      // after some row
                if (p.window != 0) look(span.low - pos0, span.low + p.rows - 1 - pos0);           // before some window
                apart = __any_sync(0xFFFFFFFFu, bad);
            }
            auto split = [&](int s, uint32_t(&ph)[4], uint32_t(&pl)[4]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    split_bf16(pr[s][h][0], pr[s][h][1], ph[h], pl[h]);
                    split_bf16(pr[s][h][2], pr[s][h][3], ph[h + 2], pl[h + 2]);
                }
            };
            if (!apart) {
                // eight outputs at a time, so that a product waits for none of the seven before it, and with the
                // fragments of the next eight on their way
                constexpr int kBlocks = kTiles * (D / 64);
                auto load_values = [&](int blk, uint32_t(&b)[4][4]) {
                    const uint32_t at = vst + (blk % (D / 64)) * (kStep * 128) + (blk / (D / 64)) * (16 * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k) ldmatrix_x4_trans(at + v_at[k], b[k][0], b[k][1], b[k][2], b[k][3]);
                };
                uint32_t vb[kAhead + 1][4][4], ph[4], pl[4];
                if constexpr (kAhead) load_values(0, vb[0]);
#pragma unroll
                for (int blk = 0; blk < kBlocks; ++blk) {
                    const int n0 = blk % (D / 64) * 8;
                    const uint32_t(&b)[4][4] = vb[blk & kAhead];
                    if (blk + kAhead < kBlocks) load_values(blk + kAhead, vb[(blk + 1) & kAhead]);
                    if (n0 == 0) split(blk / (D / 64), ph, pl);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mma_bf16(o[n0 + 2 * k], ph, b[k][0], b[k][1]);
                        mma_bf16(o[n0 + 2 * k + 1], ph, b[k][2], b[k][3]);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mma_bf16(o[n0 + 2 * k], pl, b[k][0], b[k][1]);
                        mma_bf16(o[n0 + 2 * k + 1], pl, b[k][2], b[k][3]);
                    }
                }
            } else {
#pragma unroll
                for (int s = 0; s < kTiles; ++s) {
                    uint32_t ph[4], pl[4];
                    split(s, ph, pl);
#pragma unroll 1
                    for (int r = 0; r < p.rows; ++r) {
                        const int rp = first_pos + r;
                        uint32_t keep[2];   // the halves of a fragment word whose position token r sees
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            keep[w] = 0u;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int pos = pos0 + s * 16 + w * 8 + quad * 2 + j;
                                const int back = rp - pos;
                                if (back >= 0 && (p.window == 0 || back < p.window || pos < p.sinks))
                                    keep[w] |= 0xFFFFu << (16 * j);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < D / 8; n += 2) {
                            uint32_t b0, b1, b2, b3;
                            ldmatrix_x4_trans(vst + v_at[(n >> 1) & 3] + (n >> 3) * (kStep * 128) + s * (16 * 128), b0, b1, b2,
                                              b3);
                            b0 &= keep[0], b2 &= keep[0], b1 &= keep[1], b3 &= keep[1];
                            float x[4] = {}, y[4] = {};
                            mma_bf16(x, ph, b0, b1);
                            mma_bf16(y, ph, b2, b3);
                            mma_bf16(x, pl, b0, b1);
                            mma_bf16(y, pl, b2, b3);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (row_pos[j >> 1] == rp) {
                                    o[n][j] += x[j];
                                    o[n + 1][j] += y[j];
                                }
                            }
                        }
                    }
                }
            }
            side_done();
        }

        // join the groups
        float sum[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] = l[h];
            sum[h] += __shfl_xor_sync(0xFFFFFFFFu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xFFFFFFFFu, sum[h], 2);
            if (kGroups > 1 && quad == 0)
                *reinterpret_cast<float2*>(s_ml + (grp * kRows + wr * 16 + h * 8 + gid) * 2) = make_float2(m[h], sum[h]);
        }
        auto store_out = [&](int r, int d, const float4& acc, float sum) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            *reinterpret_cast<uint2*>(p.out + row_offset(r, p.out_stride) + d) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        };
        const int cta = blockIdx.x;
        const bool cut = it.ua != 0 || it.ub != it.units;
        const int c0 = cut ? cta_of(it.g0, share.total, share.ctas) : cta;
        const Parts parts{p.part, p.part_ml, kRows, c0};
        if constexpr (kGroups == 1) {
            // nothing to join: every lane has its rows' final sums
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = wr * 16 + h * 8 + gid;
                if (row >= rows) continue;
                if (!cut) {
                    const float inv = sum[h] == 0.0f ? 0.0f : 1.0f / sum[h];
                    uint16_t* const dst = p.out + row_offset(row, p.out_stride) + quad * 2;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *reinterpret_cast<uint32_t*>(dst + n * 8) = pack_bf16(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
                } else {
                    const int64_t at = parts.row(cta - c0, row);
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *reinterpret_cast<float2*>(p.part + at * D + n * 8 + quad * 2) =
                            make_float2(o[n][2 * h], o[n][2 * h + 1]);
                    if (quad == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m[h], sum[h]);
                }
            }
        } else {
            // The outputs of many groups are brought to the rows' common maxima, and then only add up.
            float scale[2] = {1.0f, 1.0f};
            if constexpr (Cfg::kScaled) {
                named_barrier(1, kThreads);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = wr * 16 + h * 8 + gid;
                    float2 ml[kGroups / 4];   // a lane of the row's four looks at these groups
                    float top = -INFINITY, total = 0.0f;
#pragma unroll
                    for (int k = 0; k < kGroups / 4; ++k) {
                        ml[k] = *reinterpret_cast<const float2*>(s_ml + ((k * 4 + quad) * kRows + row) * 2);
                        top = fmaxf(top, ml[k].x);
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
                    for (int k = 0; k < kGroups / 4; ++k) total = fmaf(ml[k].y, exp2_approx(ml[k].x - ref), total);
                    total += __shfl_xor_sync(0xFFFFFFFFu, total, 1);
                    total += __shfl_xor_sync(0xFFFFFFFFu, total, 2);
                    scale[h] = exp2_approx(m[h] - ref);
                    if (grp == 0 && quad == 0) *reinterpret_cast<float2*>(s_sum + row * 2) = make_float2(top, total);
                }
            }
            // as many columns at a time as the rows leave room for
            constexpr int kCols = Cfg::kJoinCols;
            int wide = kCols;   // a power of two
            while (wide < D && 2 * wide * rows * kGroups * 4 <= Cfg::kJoinBytes) wide *= 2;
            const int per_row = wide / 4, row_shift = 31 - __clz(per_row);
#pragma unroll
            for (int col = 0; col < D; col += kCols) {
                const int in_round = col & (wide - 1);
                if (col > 0 && in_round == 0) named_barrier(1, kThreads);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = wr * 16 + h * 8 + gid;
                    if (row < rows) {
                        float* const at = s_join + (grp * rows + row) * wide + in_round + quad * 2;
#pragma unroll
                        for (int n = 0; n < kCols / 8; ++n)   // eight columns at place n ^ (row % 4): no bank conflicts
                            *reinterpret_cast<float2*>(at + (n ^ (gid & 3)) * 8) =
                                make_float2(o[col / 8 + n][2 * h] * scale[h], o[col / 8 + n][2 * h + 1] * scale[h]);
                    }
                }
                if (in_round + kCols != wide) continue;
                const int col0 = col + kCols - wide;
                named_barrier(1, kThreads);
                for (int e = threadIdx.x; e < rows * per_row; e += kThreads) {
                    const int row = e >> row_shift, d = (e & (per_row - 1)) * 4;
                    const float* const from = s_join + row * wide + (d ^ ((row & 3) << 3));
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    float2 sums;   // maximum and sum
                    if constexpr (Cfg::kScaled) {
                        sums = *reinterpret_cast<const float2*>(s_sum + row * 2);
#pragma unroll
                        for (int w = 0; w < kGroups; ++w) {
                            const float4 v = *reinterpret_cast<const float4*>(from + w * rows * wide);
                            acc.x += v.x;
                            acc.y += v.y;
                            acc.z += v.z;
                            acc.w += v.w;
                        }
                    } else {
                        float2 ml[kGroups];
                        sums = make_float2(-INFINITY, 0.0f);
#pragma unroll
                        for (int w = 0; w < kGroups; ++w) {
                            ml[w] = *reinterpret_cast<const float2*>(s_ml + (w * kRows + row) * 2);
                            sums.x = fmaxf(sums.x, ml[w].x);
                        }
                        const float ref = sums.x == -INFINITY ? 0.0f : sums.x;
#pragma unroll
                        for (int w = 0; w < kGroups; ++w) {
                            const float a = exp2_approx(ml[w].x - ref);
                            sums.y = fmaf(ml[w].y, a, sums.y);
                            const float4 v = *reinterpret_cast<const float4*>(from + w * rows * wide);
                            acc.x = fmaf(v.x, a, acc.x);
                            acc.y = fmaf(v.y, a, acc.y);
                            acc.z = fmaf(v.z, a, acc.z);
                            acc.w = fmaf(v.w, a, acc.w);
                        }
                    }
                    if (!cut) {
                        store_out(row, col0 + d, acc, sums.y);
                    } else {
                        const int64_t at = parts.row(cta - c0, row);
                        *reinterpret_cast<float4*>(p.part + at * D + col0 + d) = acc;
                        if (col0 + d == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = sums;
                    }
                }
            }
        }
        // a kernel of its own joins the parts of more than 16 rows, every row by a warp: one CTA would take as long as the
        // products
        if (RW > 1 && cut && it.ua == 0 && threadIdx.x == 0)
            p.joins[cta] = make_int4(cta_of(it.g0 + it.units - 1, share.total, share.ctas) - c0 + 1, seq, head, row0);
        named_barrier(1, kThreads);   // the join's buffers are free for the next item
    }

    if constexpr (RW == 1) named_barrier(2, Cfg::kThreads);   // the copying warps see to the joins
}

// Joins the parts of the cut heads, one row a warp.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) qmm_attention_join_kernel(const __grid_constant__ AttnParams p, int rw,
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
    const int rows = 16 * rw;
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

template <int D, int RW>
cudaError_t launch(const AttnParams& p0, int num_sms, cudaStream_t stream) {
    AttnParams p = p0;
    p.row_groups = (p.rows * p.group + 16 * RW - 1) / (16 * RW);
    // steps of the smallest unit: more than one only where all units might not fit 31 bits
    const int64_t steps = (static_cast<int64_t>(p.max_pages) << p.page_shift) / kStep + 2;
    p.min_unit = 1;
    while (steps / p.min_unit * p.seqs * p.kv_heads * p.row_groups >= (1LL << 30)) p.min_unit *= 2;
    int ctas = AttnCfg<D, RW>::kCtasPerSm * num_sms;
    if (ctas > kAttnMaxCtas) ctas = kAttnMaxCtas;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(AttnCfg<D, RW>::kThreads);
    cfg.dynamicSmemBytes = AttnCfg<D, RW>::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, qmm_attention_kernel<D, RW>, p);
    if (e != cudaSuccess || RW == 1) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * num_sms));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, qmm_attention_join_kernel<D>, p, RW, ctas);
}

template <int D, int RW>
cudaError_t configure() {
    // the register split would wait forever for registers that the launch did not get
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, qmm_attention_kernel<D, RW>);
    if (e != cudaSuccess) return e;
    if (a.numRegs < AttnCfg<D, RW>::kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(qmm_attention_kernel<D, RW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnCfg<D, RW>::kSmem);
}

template <int D>
cudaError_t configure_dim() {
    cudaError_t e = configure<D, 1>();
    if (e == cudaSuccess) e = configure<D, 2>();
    if (e == cudaSuccess) e = configure<D, 4>();
    return e;
}

template <int D>
cudaError_t launch_dim(const AttnParams& p, int num_sms, cudaStream_t stream) {
    const int rw = attn_row_warps(p.rows * p.group);
    if (rw == 1) return launch<D, 1>(p, num_sms, stream);
    return rw == 2 ? launch<D, 2>(p, num_sms, stream) : launch<D, 4>(p, num_sms, stream);
}

}  // namespace

cudaError_t configure_attention() {
    cudaError_t e = configure_dim<64>();
    if (e == cudaSuccess) e = configure_dim<128>();
    if (e == cudaSuccess) e = configure_dim<256>();
    return e;
}

cudaError_t launch_attention(int head_dim, const AttnParams& p, int num_sms, cudaStream_t stream) {
    if (head_dim == 64) return launch_dim<64>(p, num_sms, stream);
    if (head_dim == 128) return launch_dim<128>(p, num_sms, stream);
    return launch_dim<256>(p, num_sms, stream);
}

}  // namespace qmmk
