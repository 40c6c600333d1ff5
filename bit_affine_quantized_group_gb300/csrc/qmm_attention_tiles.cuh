// Attention over a paged cache for tiles of 16 query rows: the kernel of bfloat16 caches, and of caches of codes for more
// than 16 rows, where the team of a step first writes its codes into shared memory as binary16 numbers, for all row tiles
// read them: of keys the codes themselves, whose products each group's scale and bias then turn into scores, of values s c + b.
// (With fewer rows the numbers stay in registers: qmm_attention_codes.cuh.) Weights are one binary16 number: beside values of 11
// bits a second term took 3.3 us more for the form below and left its error as it was.
//
// Four sequences of up to 16,001 positions with 8 tokens each, 64 rows a cache head: 33.6 us from bfloat16, 39.1 from 8-bit and
// 38.4 from 4-bit codes, at a half and a quarter of the bytes: no kind is bound by them, but by a step's chain of products,
// softmax and products (with codes, and of numbers made before). Keys as binary16 numbers s c + b took 35.7 and 34.7 us, but where
// they lie 4 of their spreads from zero outputs were off by 0.0047 of their norm, 0.0016 of it their own rounding.
#pragma once

#include "qmm_attention_shared.cuh"
#include "qmm_codes.cuh"

namespace qmmk {

namespace {

// The computing warps form teams that take the steps in turn. Each warp of a team has all the positions of the step for
// 16 of up to 64 query rows, or with fewer row tiles a part of the positions: 32 where it can, for a step's chain of
// products, maximum and exponentials takes little longer for 32 positions than for 16. The outputs of 16 rows take D / 2
// registers of every lane, so that an SM has room for 8 computing warps: two CTAs of four, or one of eight for 256-wide
// heads.
template <int D, int RW, int BITS>
struct AttnCfg {
    static constexpr int kD = D, kBits = BITS, kRows = 16 * RW;
    static constexpr bool kInlineJoin = RW == 1, kSplitRegs = true;
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
    static constexpr int kComputeRegs = D == 256 ? 216 : BITS == 16 ? 184 : 176;
    static constexpr int kCopyRegs = D == 256 || BITS == 16 ? 72 : 80;
    static_assert(kCompute * kComputeRegs + 4 * kCopyRegs <= (kCompute + 4) * kLaunchRegs, "registers of a CTA");
    static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
    // steps of the shortest share: about as long as joining parts takes, and work for every team
    static constexpr int kShortShare = RW == 1 && D < 256 ? 4 : RW == 4 ? kTeams : 2;
    static constexpr int kRowBytes = D * BITS / 8;                 // a position's elements or codes
    static constexpr int kPairBytes = BITS == 16 ? 0 : D / 64 * 4; // a position's scales and biases, after the step's codes
    static constexpr int kSideBytes = kStep * (kRowBytes + kPairBytes);   // the keys or the values of a step
    // Every team has a ring of its own: in a common one, a team that only steps over the other's sides could take a
    // barrier's phase for one two rounds away.
    static constexpr int kJoinCols = D == 256 ? 32 : 64;           // columns of all rows that the groups join at once
    static constexpr int kJoinBytes = kGroups * 16 * RW * kJoinCols * 4;
    static constexpr bool kQueryRegs = D == 64 || (D == 128 && RW < 4);   // else the queries stay in shared memory
    static constexpr bool kAhead = D < 256 || RW < 4;              // fragments are read one product ahead
    static constexpr int kQueryBytes = 16 * D * 2;                 // of a row tile
    // Codes become binary16 numbers in tiles of a team: one for keys and one for values where there is room.
    static constexpr int kTileBytes = kStep * D * 2;
    static constexpr int kTileCount = BITS == 16 ? 0 : D == 256 ? 1 : 2;
    static constexpr int kRoom = D == 256 ? 227 * 1024 : 113 * 1024;   // of a CTA
    static constexpr int kMostSides = 12;
    static constexpr int kRowFloats = 1 + D / 64;                  // of a query row over codes: its unit, and its groups' sums
    static constexpr int kFixedBytes = kTeams * kTileCount * kTileBytes + kJoinBytes + RW * (kQueryRegs ? 0 : kQueryBytes) +
                                       (kGroups + 1) * 16 * RW * 8 + 2 * kMostSides * 8 + RW * 64 * kRowFloats + 16;
    // A slot of the ring of codes has both sides of a step.
    static constexpr int kSlotBytes = 2 * kSideBytes;
    static constexpr int kFit = (kRoom - kFixedBytes) / (kTeams * kSlotBytes);
    static constexpr int kSlots = kFit < kMostSides / 2 / kTeams ? kFit : kMostSides / 2 / kTeams;
    static constexpr int kSides = BITS == 16 ? (D == 64 ? 12 : 6) / kTeams - (D > 64 && RW == 4 ? 1 : 0) : 2 * kSlots;
    static constexpr int kRingBytes = kSides * kSideBytes;         // of a team
    // shared memory: rings, tiles, join, queries, their rows' units and sums, maxima and sums, barriers
    static constexpr int kTilesAt = kTeams * kRingBytes;
    static constexpr int kJoinAt = kTilesAt + kTeams * kTileCount * kTileBytes;
    static constexpr int kQueryAt = kJoinAt + kJoinBytes;
    static constexpr int kUnitAt = kQueryAt + (kQueryRegs ? 0 : RW * kQueryBytes);
    static constexpr int kMlAt = kUnitAt + (kQueryRegs || BITS == 16 ? 0 : RW * 64 * kRowFloats);
    static constexpr int kSumAt = kMlAt + kGroups * 16 * RW * 8;
    static constexpr int kBarsAt = kSumAt + (kScaled ? 16 * RW * 8 : 0);
    static constexpr int kLastAt = kBarsAt + 2 * kTeams * kSides * 8;
    static constexpr int kSmem = kLastAt + 16;
    static_assert((kJoin + 2) * 16 * 4 <= kJoinBytes, "the weights of a join fit its buffer");
    static_assert(kSmem <= kRoom, "shared memory of an SM");
    static_assert(kSides >= 2, "a side is copied while another is read");
    static __device__ __forceinline__ int key_place(int r, int c) { return r * kRowBytes + c * 16; }
    static __device__ __forceinline__ int value_place(int r, int c) { return r * kRowBytes + c * 16; }
};

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

// Weights a and b, at least 0, as bfloat16 pairs: their upper halves, and the rounded remainders (hi + lo is within 2^-16).
// The remainders get 2^-24 of the upper halves more, so that no weight from 2^-109 on has a lo of 0: that times an infinite
// value were NaN where the weight times it is infinite. (Below, weights of no more than 8 bits still have one.)
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
    constexpr float kLess = 1.0f - 0x1p-24f;
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    hi = __byte_perm(ua, ub, 0x7632);
    lo = pack_bf16(fmaf(__uint_as_float(ua & 0xFFFF0000u), -kLess, a), fmaf(__uint_as_float(ub & 0xFFFF0000u), -kLess, b));
}

template <int BITS>
__device__ __forceinline__ bool nonfinite_pair(uint32_t w) {
    constexpr uint32_t kLow = BITS == 16 ? 0x7F80u : 0x7C00u, kHigh = kLow << 16;   // the exponents' bits
    return (w & kLow) == kLow || (w & kHigh) == kHigh;
}

template <int BITS>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BITS == 16) mma_bf16(d, a, b0, b1);
    else mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
}

// The codes of a side as binary16 numbers, laid out as a side of bfloat16 is: keys as c, values as s c + b, each rounded once.
// By the 128 threads of a team.
template <class Cfg, bool KEYS>
__device__ __forceinline__ void widen(uint32_t side, uint32_t tile, int tid) {
    constexpr int kChunks = Cfg::kRowBytes / 16, kElems = 128 / Cfg::kBits;   // of a row; elements of a chunk
    static_assert(Cfg::kTeamWarps == 4, "a thread has every 128th chunk");
#pragma unroll
    for (int c = 0; c < kStep * kChunks / 128; ++c) {
        const int at = c * 128 + tid, row = at / kChunks, chunk = at % kChunks;
        const uint4 v = lds128(side + at * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const uint32_t pair = KEYS ? 0u : lds32(side + kStep * Cfg::kRowBytes + row * Cfg::kPairBytes + chunk * kElems / 64 * 4);
        const __half2 scale = half2_of(__byte_perm(pair, pair, 0x1010)), bias = half2_of(__byte_perm(pair, pair, 0x3232));
#pragma unroll
        for (int u = 0; u < kElems / 8; ++u) {   // eight elements each
            __half2 h[4];
            if constexpr (Cfg::kBits == 8) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    h[i] = __hsub2(half2_of(__byte_perm(w[2 * u + (i >> 1)], 0x64646464u, i & 1 ? 0x4342 : 0x4140)), half2_of(kHalf1024));
            } else {
                const uint32_t x = w[u], y = x >> 8;
                const __half2 low = half2_of(kHalf1024), high = half2_of(kHalf64);
                const uint32_t e0 = bits_of(__hsub2(half2_of(and_or(x, 0x000F000Fu, 0x64006400u)), low));    // 0, 4
                const uint32_t e1 = bits_of(__hsub2(half2_of(and_or(x, 0x00F000F0u, 0x54005400u)), high));   // 1, 5
                const uint32_t e2 = bits_of(__hsub2(half2_of(and_or(y, 0x000F000Fu, 0x64006400u)), low));    // 2, 6
                const uint32_t e3 = bits_of(__hsub2(half2_of(and_or(y, 0x00F000F0u, 0x54005400u)), high));   // 3, 7
                h[0] = half2_of(__byte_perm(e0, e1, 0x5410)), h[1] = half2_of(__byte_perm(e2, e3, 0x5410));
                h[2] = half2_of(__byte_perm(e0, e1, 0x7632)), h[3] = half2_of(__byte_perm(e2, e3, 0x7632));
            }
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = bits_of(KEYS ? h[i] : __hfma2(h[i], scale, bias));
            const int unit = chunk * (kElems / 8) + u;
            sts128(tile + (unit >> 3) * (kStep * 128) + row * 128 + (((unit & 7) ^ (row & 7)) << 4), make_uint4(r[0], r[1], r[2], r[3]));
        }
    }
}

template <int D, int RW, int BITS>
__global__ void __launch_bounds__(AttnCfg<D, RW, BITS>::kThreads, AttnCfg<D, RW, BITS>::kCtasPerSm)
    qmm_attention_kernel(const __grid_constant__ AttnParams p) {
    using Cfg = AttnCfg<D, RW, BITS>;
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
        if constexpr (BITS == 16)
            copy_share<Cfg>(p, share, ring, full, empty, s_join, reinterpret_cast<const float*>(smem), s_last, warp - Cfg::kCompute,
                            lane);
        else
            copy_codes<Cfg>(p, share, ring, full, empty, s_join, reinterpret_cast<const float*>(smem), s_last, warp - Cfg::kCompute,
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

    constexpr int kPlaces = BITS == 16 ? Cfg::kSides : Cfg::kSlots;               // of the team's ring,
    constexpr int kPlaceBytes = BITS == 16 ? Cfg::kSideBytes : Cfg::kSlotBytes;   // for a side, or both sides of a step of codes
    uint64_t* const my_full = full + team * kPlaces;
    uint64_t* const my_empty = empty + team * kPlaces;
    int slot = 0, round = 0;   // of the next place in the team's ring
    bool alive = true;
    auto side_full = [&]() -> uint32_t {
        if (alive) alive = wait_phase(&my_full[slot], round & 1, p.err, kErrFullWait);
        return ring + (team * kPlaces + slot) * kPlaceBytes;
    };
    auto side_done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&my_empty[slot]);
        if (++slot == kPlaces) {
            slot = 0;
            ++round;
        }
    };
    // The next side as the products read it, the keys' (0) or the values' (1), and the end of the reading. Codes become
    // binary16 numbers first, by the whole team.
    auto side_read = [&](int which) -> uint32_t {
        if constexpr (BITS == 16) {
            return side_full();
        } else {
            const uint32_t side = which == 0 ? side_full() : ring + (team * kPlaces + slot) * kPlaceBytes + Cfg::kSideBytes;
            const uint32_t tile = ring + Cfg::kTilesAt + (team * Cfg::kTileCount + (Cfg::kTileCount == 2 ? which : 0)) * Cfg::kTileBytes;
            // in one tile, the other side has been read; of two, a barrier has passed since this one's was
            if (Cfg::kTileCount == 1) named_barrier(4 + team, 32 * Cfg::kTeamWarps);
            if (which == 0) widen<Cfg, true>(side, tile, (warp % Cfg::kTeamWarps) * 32 + lane);
            else widen<Cfg, false>(side, tile, (warp % Cfg::kTeamWarps) * 32 + lane);
            if (which == 1) side_done();
            named_barrier(4 + team, 32 * Cfg::kTeamWarps);
            return tile;
        }
    };
    auto side_end = [&]() {
        if constexpr (BITS == 16) side_done();
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
        float unit[2] = {p.scale_log2, p.scale_log2};   // what a score of the lane's two rows counts, in powers of two
        float q_sum[2][D / 64];   // over codes: the sums of their queries, by groups of 64
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
                if constexpr (BITS != 16) {
                    uint32_t most = 0;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) most = max(most, max(magnitude(qf[kk][h]), magnitude(qf[kk][h + 2])));
                    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                    const QuerySize size(most, p.scale_log2);
                    unit[h] = size.unit;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        qf[kk][h] = size.f16(qf[kk][h]);
                        qf[kk][h + 2] = size.f16(qf[kk][h + 2]);
                    }
#pragma unroll
                    for (int g = 0; g < D / 64; ++g) {
                        float sum = 0.0f;
#pragma unroll
                        for (int kk = 4 * g; kk < 4 * g + 4; ++kk) sum += sum_f16(qf[kk][h]) + sum_f16(qf[kk][h + 2]);
                        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                        q_sum[h][g] = sum + __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                    }
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
                if constexpr (BITS != 16) {
                    uint32_t most = max(max(magnitude(v[k].x), magnitude(v[k].y)), max(magnitude(v[k].z), magnitude(v[k].w)));
#pragma unroll
                    for (int o = 1; o < D / 8; o <<= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
                    const QuerySize size(most, p.scale_log2);
                    v[k].x = size.f16(v[k].x), v[k].y = size.f16(v[k].y), v[k].z = size.f16(v[k].z), v[k].w = size.f16(v[k].w);
                    float* const of_row = reinterpret_cast<float*>(smem + Cfg::kUnitAt) + (wr * 16 + r) * Cfg::kRowFloats;
                    if (c == 0 && r < 16) of_row[0] = size.unit;
                    float sum = (sum_f16(v[k].x) + sum_f16(v[k].y)) + (sum_f16(v[k].z) + sum_f16(v[k].w));
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    if (c % 8 == 0 && r < 16) of_row[1 + c / 8] = sum;
                }
                if (r < 16) sts128(q_smem + r * (D * 2) + ((c ^ (r & 7)) << 4), v[k]);
            }
            named_barrier(1, kThreads);
            if constexpr (BITS != 16) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float* const of_row = reinterpret_cast<const float*>(smem + Cfg::kUnitAt) + (wr * 16 + h * 8 + gid) * Cfg::kRowFloats;
                    unit[h] = of_row[0];
#pragma unroll
                    for (int g = 0; g < D / 64; ++g) q_sum[h][g] = of_row[1 + g];
                }
            }
        }

        float o[D / 8][4];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][j] = 0.0f;

        for (int i = team; i < it.steps; i += Cfg::kTeams) {
            const int pos0 = span.step_pos(it.t0 + i) + part * kPartRows;   // the warp's first position
            const uint32_t kst = side_read(0);

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
            if constexpr (BITS == 16) {
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
                        mma<BITS>(sc[kk % kChains][2 * s], qa[kk & kAhead], b[0], b[1]);
                        mma<BITS>(sc[kk % kChains][2 * s + 1], qa[kk & kAhead], b[2], b[3]);
                    }
                }
            } else {
                // Products of the codes, two tiles at a time; each group of 64 then adds s (sum q f c) + b sum q f in float32, so that
                // keys are not rounded: those far from zero, of which only differences count, would lose the differences.
                constexpr int kPair = 2;
                static_assert(kTiles % kPair == 0 && kChains == 1, "tiles by twos");
                const uint32_t pairs = ring + (team * kPlaces + slot) * kPlaceBytes + kStep * Cfg::kRowBytes +
                                       (part * kPartRows + quad * 2) * Cfg::kPairBytes;
#pragma unroll
                for (int s0 = 0; s0 < kTiles; s0 += kPair) {
                    uint32_t kb[kAhead + 1][kPair][4], qa[kAhead + 1][4];
                    auto load_pair = [&](int kk, uint32_t(&b)[kPair][4]) {
#pragma unroll
                        for (int s = 0; s < kPair; ++s)
                            ldmatrix_x4(kst + k_at[kk & 3] + (kk >> 2) * (kStep * 128) + (s0 + s) * (16 * 128), b[s][0], b[s][1], b[s][2],
                                        b[s][3]);
                    };
                    if constexpr (kAhead) {
                        load_pair(0, kb[0]);
                        load_query(0, qa[0]);
                    }
                    float sum[2 * kPair][4];   // of a group
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        if (kk + kAhead < D / 16) {
                            load_pair(kk + kAhead, kb[(kk + 1) & kAhead]);
                            load_query(kk + kAhead, qa[(kk + 1) & kAhead]);
                        }
                        const uint32_t(&q)[4] = qa[kk & kAhead];
#pragma unroll
                        for (int n = 0; n < 2 * kPair; ++n) {
                            const uint32_t(&b)[4] = kb[kk & kAhead][n >> 1];
                            if (kk % 4 == 0) mma_f16_zc(sum[n], q[0], q[1], q[2], q[3], b[2 * (n & 1)], b[2 * (n & 1) + 1]);
                            else mma_f16(sum[n], q[0], q[1], q[2], q[3], b[2 * (n & 1)], b[2 * (n & 1) + 1]);
                        }
                        if (kk % 4 != 3) continue;
#pragma unroll
                        for (int n = 0; n < 2 * kPair; ++n) {   // positions 2 quad and 2 quad + 1 of eight
                            const uint32_t at = pairs + (s0 * 16 + n * 8) * Cfg::kPairBytes + kk / 4 * 4;
                            const float2 first = __half22float2(half2_of(lds32(at))), second = __half22float2(half2_of(lds32(at + Cfg::kPairBytes)));
                            float(&x)[4] = sc[0][2 * s0 + n];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float of_row = q_sum[h][kk / 4];
                                fma_x2(x[2 * h], x[2 * h + 1], first.y, second.y, of_row, of_row, x[2 * h], x[2 * h + 1]);
                                fma_x2(x[2 * h], x[2 * h + 1], sum[n][2 * h], sum[n][2 * h + 1], first.x, second.x, x[2 * h], x[2 * h + 1]);
                            }
                        }
                    }
                }
            }
            side_end();

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
                // scale_log2 is not negative (the queries take its sign), so that it keeps the order. Of codes the maximum is one
                // of scores before their unit: no weight passes 2^15 then, however large the scores.
                const float m_new = fmaxf(m[h], BITS != 16 || top == -INFINITY ? top : top * unit[h]);
                const float ref = m_new == -INFINITY ? 0.0f : m_new;
                alpha[h] = m_new == m[h] ? 1.0f : exp2_approx(BITS == 16 ? m[h] - ref : (m[h] - ref) * unit[h]);
                m[h] = m_new;
                float sum = 0.0f;
#pragma unroll
                for (int s = 0; s < kTiles; ++s) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = pr[s][h][j];
                        pr[s][h][j] = exp2_approx(BITS == 16 ? fmaf(x, unit[h], -ref) : fmaf(x - ref, unit[h], kWeightBits));
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

            const uint32_t vst = side_read(1);
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
                        bad |= nonfinite_pair<BITS>(w.x) || nonfinite_pair<BITS>(w.y) || nonfinite_pair<BITS>(w.z) || nonfinite_pair<BITS>(w.w);
                    }
                };
                look(first_pos + 1 - pos0, seq_end() - pos0);                                      // after some row
                if (p.window != 0) look(span.low - pos0, span.low + p.rows - 1 - pos0);           // before some window
                apart = __any_sync(0xFFFFFFFFu, bad);
            }
            auto split = [&](int s, uint32_t(&ph)[4], uint32_t(&pl)[4]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (BITS == 16) {
                        split_bf16(pr[s][h][0], pr[s][h][1], ph[h], pl[h]);
                        split_bf16(pr[s][h][2], pr[s][h][3], ph[h + 2], pl[h + 2]);
                    } else {
                        ph[h] = pack_f16(pr[s][h][0], pr[s][h][1]);
                        ph[h + 2] = pack_f16(pr[s][h][2], pr[s][h][3]);
                    }
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
                        mma<BITS>(o[n0 + 2 * k], ph, b[k][0], b[k][1]);
                        mma<BITS>(o[n0 + 2 * k + 1], ph, b[k][2], b[k][3]);
                    }
                    if constexpr (BITS == 16) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma<BITS>(o[n0 + 2 * k], pl, b[k][0], b[k][1]);
                            mma<BITS>(o[n0 + 2 * k + 1], pl, b[k][2], b[k][3]);
                        }
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
                            mma<BITS>(x, ph, b0, b1);
                            mma<BITS>(y, ph, b2, b3);
                            if constexpr (BITS == 16) {
                                mma<BITS>(x, pl, b0, b1);
                                mma<BITS>(y, pl, b2, b3);
                            }
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
            side_end();
        }

        // join the groups
        float sum[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] = l[h];
            if constexpr (BITS != 16) m[h] *= unit[h];
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

template <int D, int RW, int BITS>
cudaError_t launch_tiles(const AttnParams& p, int num_sms, cudaStream_t stream) {
    return launch<AttnCfg<D, RW, BITS>>(qmm_attention_kernel<D, RW, BITS>, p, num_sms, stream);
}

template <int D, int RW, int BITS>
cudaError_t configure_tiles() {
    return configure<AttnCfg<D, RW, BITS>>(qmm_attention_kernel<D, RW, BITS>);
}

}  // namespace

}  // namespace qmmk
