// Attention over a paged cache of 8- or 4-bit codes for up to 16 query rows of a cache head.
//
// The products are transposed, so that codes are their left operands and tiles of 8 query rows their right ones:
//   S^T = K Q^T,   O^T = V^T P^T.
// Scores of a lane are those of a position and two rows; two of them packed to binary16 and transposed across the warp
// (movmatrix) are the second product's operand. The codes of a step stay in registers between shared memory and product:
//   - A key's codes c become binary16 numbers 1024 + c (by a byte permutation, two at a time; of 4-bit codes half become
//     64 + c, by masks), the queries q f with a power of two f of their row. A group of 64 elements adds
//       s (sum q f (1024 + c) - 1024 sum q f) + b sum q f
//     to f times the score, in float32.
//   - A value's code becomes the binary16 number c 2^-24 (c 2^-20 of 4 bits), which has no offset to take off again; its scale
//     goes into the weight, P s, for each group of 64 columns; the biases are one more product of the weights themselves:
//     O = 2^24 sum (P s) (c 2^-24) + sum P b.
//   - The tensor cores cut what they add at about 2^-24 of the largest term, always to the same side, and a subnormal number
//     counts as one of 2^-14. Where codes and biases cancel, sums of all steps kept there lost more the longer the sequence was;
//     so only a step's are, and the steps are added up by float32 additions, which round. 4-bit codes are held as high as a
//     nibble's place allows for the same reason.
//   - The weights P are two binary16 terms, the first of up to 2^15 (4 bits: 2^13), so that with scales below 2 (8) P s is as well:
//     two products, as in the kernel of bfloat16 caches, for one term rounds values that cancel by more than the output's own
//     rounding. Larger scales take the values themselves, s c + b rounded once.
//
// What bounds it: with 8-bit codes bytes, with 4-bit codes the computing warps, of which registers allow two a scheduler, with
// a step's chain of products, maximum, exponentials, transposition and products. One sequence of 131,072 positions with 8 heads
// of 128: 54.5 us with 8 bits (5.2 TB/s), 51.3 with 4 (2.9 TB/s); 64 ragged sequences: 122 us (4.9 TB/s) and 116. About 7 us of
// each are start and join. (Weights of one term: 54.7, 48.5, 117 and 110; sums of all steps in the tensor cores besides: 52.4, 44.6,
// 114 and 102. Added late, with the next step's: no gain; begun with the biases' products: 53.5 and 121 of 4 bits.) A branch
// that the compiler does not know to be the whole warp's costs: masks in one block for all rows, one for the slow path and votes
// before both took 48.1 us of 4 bits to 44.9. Tried before all that, in us of the two long forms of 4 bits (then 48 and 111): values
// as numbers, by a multiply-add each, the same; a step's key products before the last one's softmax 59 and 127; 12 computing warps
// in one CTA 52 and 158; four warps a step slower in both, one warp a step 47 and 120. Codes made numbers in shared memory first,
// as for more rows, took 82.
#pragma once

#include <type_traits>

#include "qmm_attention_shared.cuh"
#include "qmm_attention_tiles.cuh"
#include "qmm_codes.cuh"

namespace qmmk {

namespace {

// ROWS8: tiles of 8 query rows, 1 or 2. Warps take parts of a step's positions, so that each has all rows.
template <int D, int ROWS8, int BITS>
struct CodesCfg {
    static constexpr int kD = D, kBits = BITS, kRows = 8 * ROWS8;
    static constexpr bool kInlineJoin = true, kSplitRegs = true;
    static constexpr int kCompute = D == 256 ? 8 : 4;              // computing warps
    static constexpr int kTeamWarps = D == 256 ? 4 : 2;
    static constexpr int kTeams = kCompute / kTeamWarps;
    static constexpr int kTiles = 4 / kTeamWarps;                  // 16-position tiles of a warp
    static constexpr int kThreads = 32 * (kCompute + 4);           // and a group of four that starts the copies
    static constexpr int kLaunchRegs = D == 256 ? 168 : 128;
    // (heads of 128 in 152 and 104: 64 ragged sequences of 8 bits a twelfth slower)
    static constexpr int kComputeRegs = D == 256 ? (ROWS8 == 1 ? 200 : 216) : D == 64 && ROWS8 == 1 ? 152 : 176;
    static constexpr int kCopyRegs = ROWS8 == 1 && D != 128 ? 104 : D == 256 ? 72 : 80;
    static_assert(kCompute * kComputeRegs + 4 * kCopyRegs <= (kCompute + 4) * kLaunchRegs, "registers of a CTA");
    static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
    static constexpr int kShortShare = D < 256 ? 4 : 2;            // steps of the shortest share
    static constexpr int kRowBytes = D * BITS / 8;                 // a position's codes
    static constexpr int kPairBytes = D / 64 * 4;                  // its scales and biases, after the step's codes
    static constexpr int kSideBytes = kStep * (kRowBytes + kPairBytes);
    static constexpr int kJoinCols = D == 256 && ROWS8 == 2 ? 32 : 64;   // columns of all rows that the warps join at once
    static constexpr int kJoinBytes = kCompute * kRows * kJoinCols * 4;
    // Weights are binary16 terms of up to 2^kWeightBits. Times a scale of up to kMostScale (2 or 8, as a binary16 number) they
    // still are.
    static constexpr float kWeightBits = BITS == 8 ? 15.0f : 13.0f;
    static constexpr uint32_t kMostScale = BITS == 8 ? 0x3FFFu : 0x47FFu;
    static constexpr float kUnit = BITS == 8 ? 0x1p24f : 0x1p20f;  // what products with codes count by
    static constexpr bool kQueryRegs = D < 256;                    // else the queries stay in shared memory
    static constexpr int kQueryBytes = kQueryRegs ? 0 : D * kRows * 2;
    static constexpr int kSumBytes = kRows * (D / 64 * 8 + 4);     // of the queries' groups, and their rows' units
    static constexpr int kSums = kQueryRegs ? kCompute : 1;        // each warp has its own, or all the same
    static constexpr int kRoom = D == 256 ? 227 * 1024 : 113 * 1024;   // of a CTA
    static constexpr int kSlotBytes = 2 * kSideBytes;              // both sides of a step
    static constexpr int kMostSlots = 8;                           // of all teams
    static constexpr int kFixedBytes = kJoinBytes + kQueryBytes + kSums * kSumBytes + (kCompute + 1) * kRows * 8 + 2 * kMostSlots * 8 + 16;
    static constexpr int kFit = (kRoom - kFixedBytes) / (kTeams * kSlotBytes);
    static constexpr int kSlots = kFit < kMostSlots / kTeams ? kFit : kMostSlots / kTeams;
    static constexpr int kRingBytes = kSlots * kSlotBytes;         // of a team
    static constexpr int kJoinAt = kTeams * kRingBytes;
    static constexpr int kQueryAt = kJoinAt + kJoinBytes;
    static constexpr int kSumsAt = kQueryAt + kQueryBytes;
    static constexpr int kMlAt = kSumsAt + kSums * kSumBytes;
    static constexpr int kTotalAt = kMlAt + kCompute * kRows * 8;
    static constexpr int kBarsAt = kTotalAt + kRows * 8;
    static constexpr int kLastAt = kBarsAt + 2 * kTeams * kSlots * 8;
    static constexpr int kSmem = kLastAt + 16;
    static_assert((kJoin + 2) * kRows * 4 <= kJoinBytes, "the weights of a join fit its buffer");
    static_assert(kSmem <= kRoom && kSlots >= 2, "shared memory of an SM");
    static_assert(kSideBytes % 128 == 0 && kSumBytes % 16 == 0 && kMlAt % 16 == 0 && kBarsAt % 8 == 0, "alignment");

    // Codes in a side: the 16-byte chunk c of the position r of a tile of 16, by rows of positions for keys and with the
    // even and the odd positions of eight apart for values, so that the vectors that a warp reads at once lie in
    // different banks.
    static constexpr int kChunks = kRowBytes / 16;
    static __device__ __forceinline__ int key_place(int r, int c) {
        const int x = BITS == 8 ? (kChunks >= 8 ? (r & 1) << 2 : 0) : kChunks == 8 ? (r & 3) << 1 : kChunks == 4 ? r & 2 : 0;
        return r * kRowBytes + ((c ^ x) << 4);
    }
    static __device__ __forceinline__ int value_place(int r, int c) {
        const int slot = (r & 8) | ((r & 1) << 2) | ((r >> 1) & 3);
        const int x = kChunks >= 8 ? (slot & 3) << 1 : kChunks == 4 ? slot & 2 : 0;
        return slot * kRowBytes + ((c ^ x) << 4);
    }
};

// Transposes an 8 x 8 matrix of 16-bit elements, two neighbours of a row in each lane.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// d = a b + c, with c the same for both rows of a lane
__device__ __forceinline__ void mma_f16_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// The places among a lane's 16 neighbours of a group of the elements i = 0..3 of its fragment of the product w = 0..3: two
// in the first half and two in the second. 4-bit codes come from a word's nibbles k and k + 4.
template <int BITS>
__device__ __forceinline__ constexpr int element_of(int w, int i) {
    if (BITS == 8) return 4 * w + i;
    return 8 * (w >> 1) + 2 * (w & 1) + (i & 1) * 4 + (i >> 1);
}

// The two halves of product w's fragment from a lane's codes of 16 neighbours: 1024 + c; of 4-bit codes 64 + c in the second.
template <int BITS>
__device__ __forceinline__ void key_fragment(const uint32_t (&codes)[BITS / 2], int w, uint32_t& first, uint32_t& second) {
    if constexpr (BITS == 8) {
        first = __byte_perm(codes[w], 0x64646464u, 0x4140);
        second = __byte_perm(codes[w], 0x64646464u, 0x4342);
    } else {
        const uint32_t x = w & 1 ? codes[w >> 1] >> 8 : codes[w >> 1];
        first = and_or(x, 0x000F000Fu, kHalf1024);
        second = and_or(x, 0x00F000F0u, kHalf64);
    }
}

// The codes of four neighbouring columns of two positions, from their words: pairs over the positions, as binary16 numbers
// c 2^-24, or c 2^-20 of 4 bits. quarter: of a word of 4-bit codes, its half.
template <int BITS>
__device__ __forceinline__ void code_pairs(uint32_t first, uint32_t second, int quarter, uint32_t (&v)[4]) {
    if constexpr (BITS == 8) {
        const uint32_t x = __byte_perm(first, second, 0x5140), y = __byte_perm(first, second, 0x7362);
        v[0] = __byte_perm(x, 0u, 0x4140);
        v[1] = __byte_perm(x, 0u, 0x4342);
        v[2] = __byte_perm(y, 0u, 0x4140);
        v[3] = __byte_perm(y, 0u, 0x4342);
    } else {
        const uint32_t x = __byte_perm(first, second, quarter == 0 ? 0x5410 : 0x7632);
        v[0] = (x << 4) & 0x00F000F0u;
        v[1] = x & 0x00F000F0u;
        v[2] = (x >> 4) & 0x00F000F0u;
        v[3] = (x >> 8) & 0x00F000F0u;
    }
}

// The same as values, s c + b rounded once.
template <int BITS>
__device__ __forceinline__ void value_pairs(uint32_t first, uint32_t second, int quarter, uint32_t scale, uint32_t bias, uint32_t (&v)[4]) {
    constexpr uint32_t kZero = BITS == 8 ? kHalf1024 : kHalf64;   // the number whose last bits the code's are
    code_pairs<BITS>(first, second, quarter, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bits_of(__hfma2(__hsub2(half2_of(v[i] | kZero), half2_of(kZero)), half2_of(scale), half2_of(bias)));
}

template <int D, int ROWS8, int BITS>
__global__ void __launch_bounds__(CodesCfg<D, ROWS8, BITS>::kThreads, CodesCfg<D, ROWS8, BITS>::kCtasPerSm)
    qmm_attention_codes_kernel(const __grid_constant__ AttnParams p) {
    using Cfg = CodesCfg<D, ROWS8, BITS>;
    constexpr int kRows = Cfg::kRows;              // query rows of a CTA
    constexpr int kTiles = Cfg::kTiles;
    constexpr int kPartRows = 16 * kTiles;         // positions of a warp's part of a step
    constexpr int kThreads = 32 * Cfg::kCompute;   // computing threads
    constexpr int kGroups = D / 64;
    constexpr int kEach = 8;                       // neighbouring columns of a lane in each group of 64
    constexpr int kSets = D / 64;
    constexpr int kBiases = kSets < 2 ? 1 : kSets / 2;   // products of two groups' biases
    constexpr int kPairsAt = kStep * Cfg::kRowBytes;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* const full = reinterpret_cast<uint64_t*>(smem + Cfg::kBarsAt);
    uint64_t* const empty = full + Cfg::kTeams * Cfg::kSlots;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(smem);
    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::kTeams * Cfg::kSlots; ++i) {
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
    if (!any) return;
    if (warp >= Cfg::kCompute) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kCopyRegs));
        copy_codes<Cfg>(p, share, ring, full, empty, s_join, reinterpret_cast<const float*>(smem), s_last, warp - Cfg::kCompute, lane);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kComputeRegs));

    const int team = warp / Cfg::kTeamWarps;    // takes the steps team, team + kTeams, ... of every item
    const int part = warp % Cfg::kTeamWarps;    // its part of the step's positions
    const int quad = lane & 3, gid = lane >> 2;
    const uint32_t q_smem = ring + Cfg::kQueryAt;
    uint8_t* const sums = smem + Cfg::kSumsAt + (Cfg::kQueryRegs ? warp * Cfg::kSumBytes : 0);   // [group][row] two floats
    float* const units = reinterpret_cast<float*>(sums + kRows * kGroups * 8);
    float* const s_ml = reinterpret_cast<float*>(smem + Cfg::kMlAt);           // [warp][row][2]
    float* const s_total = reinterpret_cast<float*>(smem + Cfg::kTotalAt);     // [row][2]

    // What a lane reads of a slot, of which all else lies at fixed distances: its chunks of the position gid of each group of
    // keys, its columns of the position 2 quad of values, and their positions' scales and biases.
    uint32_t key_at[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
        key_at[k] = part * kPartRows * Cfg::kRowBytes +
                    (BITS == 8 ? Cfg::key_place(gid, 4 * k + quad) : Cfg::key_place(gid, 2 * k + (quad >> 1)) + (quad & 1) * 8);
    uint32_t value_at[kSets];
#pragma unroll
    for (int c = 0; c < kSets; ++c) {
        const int byte = (c * 8 + gid) * kEach * BITS / 8;
        value_at[c] = Cfg::kSideBytes + part * kPartRows * Cfg::kRowBytes + Cfg::value_place(2 * quad, byte >> 4) + (byte & 15);
    }
    const uint32_t key_pair_at = kPairsAt + (part * kPartRows + gid) * Cfg::kPairBytes;
    const uint32_t value_pair_at = Cfg::kSideBytes + kPairsAt + (part * kPartRows + 2 * quad) * Cfg::kPairBytes;

    uint64_t* const my_full = full + team * Cfg::kSlots;
    uint64_t* const my_empty = empty + team * Cfg::kSlots;
    int slot = 0, round = 0;   // of the next step in the team's ring
    bool alive = true;
    auto slot_full = [&]() -> uint32_t {
        if (alive) alive = wait_phase(&my_full[slot], round & 1, p.err, kErrFullWait);
        return ring + (team * Cfg::kSlots + slot) * Cfg::kSlotBytes;
    };
    auto slot_done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&my_empty[slot]);
        if (++slot == Cfg::kSlots) {
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
        // The queries' fragments: a lane has 16 neighbours of every group of 64 elements of the row gid of each tile.
        uint32_t qf[Cfg::kQueryRegs ? D / 16 : 1][ROWS8][2];
        if (Cfg::kQueryRegs || warp == 0) {   // all warps have the same rows
            __syncwarp();   // the last item's sums have been read
#pragma unroll
            for (int n = 0; n < ROWS8; ++n) {
                const int i = n * 8 + gid;
                const bool in = i < rows;
                const uint16_t* src = p.q + (in ? row_offset(i, p.q_stride) : 0) + quad * 16;
                uint32_t w[kGroups][8];
                uint32_t most = 0;
#pragma unroll
                for (int k = 0; k < kGroups; ++k) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (in) v = *reinterpret_cast<const uint4*>(src + k * 64 + j * 8);
                        w[k][4 * j] = v.x, w[k][4 * j + 1] = v.y, w[k][4 * j + 2] = v.z, w[k][4 * j + 3] = v.w;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        w[k][j] ^= p.query_sign;
                        most = max(most, magnitude(w[k][j]));
                    }
                }
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                const QuerySize size(most, p.scale_log2);
#pragma unroll
                for (int k = 0; k < kGroups; ++k) {
                    float sum = 0.0f, more = 0.0f;   // of q f, and of q f times 1024 or 64
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float e[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int at = element_of<BITS>(j, x);
                            e[x] = __uint_as_float(at & 1 ? w[k][at >> 1] & 0xFFFF0000u : w[k][at >> 1] << 16) * size.factor;
                        }
                        const uint32_t a = pack_f16(e[0], e[1]), b = pack_f16(e[2], e[3]);
                        const float2 fa = __half22float2(half2_of(a)), fb = __half22float2(half2_of(b));
                        const float low = fa.x + fa.y, high = fb.x + fb.y;
                        sum += low + high;
                        more += 1024.0f * low + (BITS == 8 ? 1024.0f : 64.0f) * high;
                        if constexpr (Cfg::kQueryRegs) {
                            qf[k * 4 + j][n][0] = a;
                            qf[k * 4 + j][n][1] = b;
                        } else {
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(q_smem + ((n * (D / 16) + k * 4 + j) * 32 + lane) * 8),
                                         "r"(a), "r"(b) : "memory");
                        }
                    }
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                        more += __shfl_xor_sync(0xFFFFFFFFu, more, o);
                    }
                    if (quad == 0) *reinterpret_cast<float2*>(sums + (k * kRows + i) * 8) = make_float2(sum, more);
                }
                if (quad == 0) units[i] = size.unit;
            }
            __syncwarp();
        }
        if constexpr (!Cfg::kQueryRegs) named_barrier(1, kThreads);
        // of the lane's two rows 2 quad and 2 quad + 1 of each tile
        float unit[ROWS8][2], m[ROWS8][2], l[ROWS8][2];
        int row_pos[ROWS8][2];   // their positions; -1 for none
#pragma unroll
        for (int n = 0; n < ROWS8; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = n * 8 + quad * 2 + j;
                unit[n][j] = units[i];
                row_pos[n][j] = i < rows ? first_pos + token_of(i) : -1;
                m[n][j] = -INFINITY;
                l[n][j] = 0.0f;
            }

        float o[D / 16][ROWS8][4], ob[kBiases][ROWS8][4];   // columns by rows of scaled codes; of biases, two groups of 64
#pragma unroll
        for (int n = 0; n < ROWS8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c) o[c][n][j] = 0.0f;
#pragma unroll
                for (int c = 0; c < kBiases; ++c) ob[c][n][j] = 0.0f;
            }

        for (int i = team; i < it.steps; i += Cfg::kTeams) {
            const int pos0 = span.step_pos(it.t0 + i) + part * kPartRows;   // the warp's first position
            float sc[kTiles][ROWS8][4];   // [tile][rows][position gid or gid + 8, row]
#pragma unroll
            for (int s = 0; s < kTiles; ++s)
#pragma unroll
                for (int n = 0; n < ROWS8; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[s][n][j] = 0.0f;
            const uint32_t side = slot_full();
            // positions that every row sees need no mask (the vote tells the compiler that the warp takes one way)
            const bool whole = __all_sync(
                0xFFFFFFFFu, pos0 + kPartRows <= min(first_pos + 1, p.positions) &&
                                 (p.window == 0 || first_pos + p.rows - 1 - pos0 < p.window || pos0 + kPartRows <= p.sinks));
            // Scales that weights leave binary16 with, infinities and NaN take a slow path: the values themselves, and for each
            // token's rows a product of their own without what they do not see, for a position that only some rows see weighs
            // nothing in the others, but 0 * inf is not 0.
            bool slow = false;
#pragma unroll
            for (int c = 0; c < kPartRows * kGroups; c += 32) {
                if (kPartRows * kGroups < 32 && lane >= kPartRows * kGroups) break;
                const uint32_t pair = lds32(side + (Cfg::kSideBytes + kPairsAt + part * kPartRows * Cfg::kPairBytes) + (c + lane) * 4);
                slow |= (pair & 0x7FFFu) > Cfg::kMostScale;
                slow |= (pair & 0x7FFF0000u) >= 0x7C000000u;   // the bias
            }
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                float part_sc[kTiles][ROWS8][4];
                uint4 q_sums[ROWS8];   // sum and more of the two rows
#pragma unroll
                for (int n = 0; n < ROWS8; ++n) q_sums[n] = *reinterpret_cast<const uint4*>(sums + (k * kRows + n * 8 + quad * 2) * 8);
#pragma unroll
                for (int s = 0; s < kTiles; ++s) {
                    uint32_t codes[2][BITS / 2];   // of positions gid and gid + 8
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t at = side + key_at[k] + (s * 16 + h * 8) * Cfg::kRowBytes;
                        if constexpr (BITS == 8) {
                            const uint4 v = lds128(at);
                            codes[h][0] = v.x, codes[h][1] = v.y, codes[h][2] = v.z, codes[h][3] = v.w;
                        } else {
                            const uint2 v = lds64(at);
                            codes[h][0] = v.x, codes[h][1] = v.y;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a[4];
                        key_fragment<BITS>(codes[0], w, a[0], a[2]);
                        key_fragment<BITS>(codes[1], w, a[1], a[3]);
#pragma unroll
                        for (int n = 0; n < ROWS8; ++n) {
                            uint32_t b0, b1;
                            if constexpr (Cfg::kQueryRegs) {
                                b0 = qf[k * 4 + w][n][0], b1 = qf[k * 4 + w][n][1];
                            } else {
                                const uint2 v = lds64(q_smem + ((n * (D / 16) + k * 4 + w) * 32 + lane) * 8);
                                b0 = v.x, b1 = v.y;
                            }
                            if (w == 0) mma_f16_from(part_sc[s][n], a, b0, b1, -__uint_as_float(q_sums[n].y), -__uint_as_float(q_sums[n].w));
                            else mma_f16(part_sc[s][n], a[0], a[1], a[2], a[3], b0, b1);
                        }
                    }
                }
#pragma unroll
                for (int s = 0; s < kTiles; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 sb = __half22float2(half2_of(lds32(side + key_pair_at + (s * 16 + h * 8) * Cfg::kPairBytes + k * 4)));
#pragma unroll
                        for (int n = 0; n < ROWS8; ++n) {
                            float(&x)[4] = sc[s][n];
                            const float(&a)[4] = part_sc[s][n];
                            x[2 * h] = fmaf(sb.x, a[2 * h], fmaf(sb.y, __uint_as_float(q_sums[n].x), x[2 * h]));
                            x[2 * h + 1] = fmaf(sb.x, a[2 * h + 1], fmaf(sb.y, __uint_as_float(q_sums[n].z), x[2 * h + 1]));
                        }
                    }
            }
            if (!whole) {
#pragma unroll
                for (int n = 0; n < ROWS8; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // position s * 16 + h * 8 of the lane's lies after its row or the table's end, or before the window
                        // and past the sinks
                        const int own = row_pos[n][j] - pos0 - gid;
                        const int last = min(own, seq_end() - 1 - pos0 - gid);
                        // (in 32 bits without a sign: wraps for rows without a position, which see nothing anyway)
                        const int out = p.window == 0 ? -1 : static_cast<int>(static_cast<uint32_t>(own) - p.window);
                        const int sink = p.window == 0 ? -1 : p.sinks - pos0 - gid;
#pragma unroll
                        for (int s = 0; s < kTiles; ++s)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int at = s * 16 + h * 8;
                                if (at > last || (at <= out && at >= sink)) sc[s][n][2 * h + j] = -INFINITY;
                            }
                    }
            }
            float alpha[ROWS8][2];
            bool same = true;
#pragma unroll
            for (int n = 0; n < ROWS8; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = -INFINITY;
#pragma unroll
                    for (int s = 0; s < kTiles; ++s) top = fmaxf(top, fmaxf(sc[s][n][j], sc[s][n][2 + j]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                    // The maximum is one of scores before their unit, which is above 0 and keeps the order: a difference to it
                    // is exact to a rounding of its own, so that no weight passes its bits, and becomes an infinity, however large
                    // the scores.
                    const float m_new = fmaxf(m[n][j], top);
                    const float ref = m_new == -INFINITY ? 0.0f : m_new;
                    alpha[n][j] = exp2_approx((m[n][j] - ref) * unit[n][j]);
                    same &= m_new == m[n][j];
                    m[n][j] = m_new;
                    float sum = 0.0f;
#pragma unroll
                    for (int s = 0; s < kTiles; ++s) {
                        float &x = sc[s][n][j], &y = sc[s][n][2 + j];
                        add_x2(x, y, x, y, -ref, -ref);
                        fma_x2(x, y, x, y, unit[n][j], unit[n][j], Cfg::kWeightBits, Cfg::kWeightBits);
                        x = exp2_approx(x), y = exp2_approx(y);
                        sum += x;
                        sum += y;
                    }
                    l[n][j] = fmaf(l[n][j], alpha[n][j], sum);
                }
            slow = __any_sync(0xFFFFFFFFu, slow);
            if (__any_sync(0xFFFFFFFFu, !same)) {
#pragma unroll
                for (int n = 0; n < ROWS8; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) o[c][n][j] *= alpha[n][j & 1];
#pragma unroll
                        for (int c = 0; c < kBiases; ++c) ob[c][n][j] *= alpha[n][j & 1];
                    }
            }

            uint32_t pb[kTiles][ROWS8][2], pl[kTiles][ROWS8][2];   // the weights' terms, as right operands
#pragma unroll
            for (int s = 0; s < kTiles; ++s)
#pragma unroll
                for (int n = 0; n < ROWS8; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        split_f16(sc[s][n][2 * h], sc[s][n][2 * h + 1], pb[s][n][h], pl[s][n][h]);
                        pb[s][n][h] = transposed(pb[s][n][h]);
                        pl[s][n][h] = transposed(pl[s][n][h]);
                    }
            auto load_pairs = [&](int s, uint32_t (&pairs)[4][kSets]) {   // of a tile's values, positions 2 quad + {0, 1, 8, 9}
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t at = side + value_pair_at + (s * 16 + (j & 1) + (j >> 1) * 8) * Cfg::kPairBytes;
                    if constexpr (kSets == 1) {
                        pairs[j][0] = lds32(at);
                    } else if constexpr (kSets == 2) {
                        const uint2 v = lds64(at);
                        pairs[j][0] = v.x, pairs[j][1] = v.y;
                    } else {
                        const uint4 v = lds128(at);
                        pairs[j][0] = v.x, pairs[j][1] = v.y, pairs[j][2] = v.z, pairs[j][3] = v.w;
                    }
                }
            };
            auto scales = [](const uint32_t (&pairs)[4][kSets], int c, int h) { return __byte_perm(pairs[2 * h][c], pairs[2 * h + 1][c], 0x5410); };
            auto biases = [](const uint32_t (&pairs)[4][kSets], int c, int h) { return __byte_perm(pairs[2 * h][c], pairs[2 * h + 1][c], 0x7632); };
            constexpr int kWords = kEach * BITS / 32, kPerWord = 32 / BITS;   // of a lane's codes
            auto load_codes = [&](int s, int c, uint32_t (&codes)[4][kWords]) {   // of a tile's group, of those positions
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // (the odd positions of eight lie four rows behind the even ones)
                    const uint32_t at = side + value_at[c] + (s * 16 + (j & 1) * 4 + (j >> 1) * 8) * Cfg::kRowBytes;
                    if constexpr (kWords == 2) {
                        const uint2 v = lds64(at);
                        codes[j][0] = v.x, codes[j][1] = v.y;
                    } else {
                        codes[j][0] = lds32(at);
                    }
                }
            };
            if (__builtin_expect(!slow, 1)) {
                uint32_t pairs[kTiles][4][kSets];
#pragma unroll
                for (int s = 0; s < kTiles; ++s) load_pairs(s, pairs[s]);
#pragma unroll
                for (int c = 0; c < kBiases; ++c) {
                    const int other = kSets > 1 ? 2 * c + 1 : 0;
                    float sum[ROWS8][4];   // of the step
#pragma unroll
                    for (int s = 0; s < kTiles; ++s)
#pragma unroll
                        for (int n = 0; n < ROWS8; ++n) {
                            const uint32_t b[4] = {biases(pairs[s], 2 * c, 0), biases(pairs[s], other, 0), biases(pairs[s], 2 * c, 1), biases(pairs[s], other, 1)};
                            if (s == 0) mma_f16_zc(sum[n], b[0], b[1], b[2], b[3], pb[s][n][0], pb[s][n][1]);
                            else mma_f16(sum[n], b[0], b[1], b[2], b[3], pb[s][n][0], pb[s][n][1]);
                            mma_f16(sum[n], b[0], b[1], b[2], b[3], pl[s][n][0], pl[s][n][1]);
                        }
#pragma unroll
                    for (int n = 0; n < ROWS8; ++n) {
                        add_x2(ob[c][n][0], ob[c][n][1], ob[c][n][0], ob[c][n][1], sum[n][0], sum[n][1]);
                        add_x2(ob[c][n][2], ob[c][n][3], ob[c][n][2], ob[c][n][3], sum[n][2], sum[n][3]);
                    }
                }
#pragma unroll
                for (int c = 0; c < kSets; ++c) {
                    float sum[kEach / 2][ROWS8][4];   // of the step: columns by rows
#pragma unroll
                    for (int s = 0; s < kTiles; ++s) {
                        uint32_t codes[4][kWords];
                        load_codes(s, c, codes);
                        uint32_t ph[ROWS8][2], pr[ROWS8][2];   // weights times scales, in two terms as well
#pragma unroll
                        for (int n = 0; n < ROWS8; ++n)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const __half2 hi = half2_of(pb[s][n][h]), of = half2_of(scales(pairs[s], c, h)), first = __hmul2(hi, of);
                                ph[n][h] = bits_of(first);
                                pr[n][h] = bits_of(__hfma2(half2_of(pl[s][n][h]), of, __hfma2(hi, of, __hneg2(first))));
                            }
#pragma unroll
                        for (int e = 0; e < kEach; e += 4) {
                            uint32_t v0[4], v1[4];
                            const int word = e / kPerWord, quarter = e % kPerWord / 4;
                            code_pairs<BITS>(codes[0][word], codes[1][word], quarter, v0);
                            code_pairs<BITS>(codes[2][word], codes[3][word], quarter, v1);
#pragma unroll
                            for (int k = 0; k < 4; k += 2)
#pragma unroll
                                for (int n = 0; n < ROWS8; ++n) {
                                    float(&to)[4] = sum[(e + k) / 2][n];
                                    if (s == 0) mma_f16_zc(to, v0[k], v0[k + 1], v1[k], v1[k + 1], ph[n][0], ph[n][1]);
                                    else mma_f16(to, v0[k], v0[k + 1], v1[k], v1[k + 1], ph[n][0], ph[n][1]);
                                }
#pragma unroll
                            for (int k = 0; k < 4; k += 2)
#pragma unroll
                                for (int n = 0; n < ROWS8; ++n)
                                    mma_f16(sum[(e + k) / 2][n], v0[k], v0[k + 1], v1[k], v1[k + 1], pr[n][0], pr[n][1]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kEach / 2; ++k)
#pragma unroll
                        for (int n = 0; n < ROWS8; ++n) {
                            float(&to)[4] = o[c * (kEach / 2) + k][n];
                            float(&x)[4] = sum[k][n];
                            add_x2(to[0], to[1], to[0], to[1], x[0], x[1]);
                            add_x2(to[2], to[3], to[2], to[3], x[2], x[3]);
                        }
                }
            } else {
                // Products of the values themselves, for the rows of one token at a time, without what they do not see.
#pragma unroll
                for (int s = 0; s < kTiles; ++s) {
                    uint32_t pairs[4][kSets];
                    load_pairs(s, pairs);
#pragma unroll
                    for (int n = 0; n < ROWS8; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) pl[s][n][h] = some_left(pb[s][n][h], pl[s][n][h]);
#pragma unroll 1
                    for (int r = 0; r < p.rows; ++r) {
                        const int rp = first_pos + r;
                        uint32_t keep[2];
#pragma unroll
                        for (int w = 0; w < 2; ++w) {   // the halves of a fragment word whose position token r sees
                            keep[w] = 0u;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int pos = pos0 + s * 16 + w * 8 + quad * 2 + j;
                                const int back = rp - pos;
                                if (back >= 0 && (p.window == 0 || back < p.window || pos < p.sinks)) keep[w] |= 0xFFFFu << (16 * j);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < kSets; ++c) {
                            uint32_t codes[4][kWords];
                            load_codes(s, c, codes);
#pragma unroll
                            for (int e = 0; e < kEach; e += 4) {
                                uint32_t v0[4], v1[4];
                                const int word = e / kPerWord, quarter = e % kPerWord / 4;
                                value_pairs<BITS>(codes[0][word], codes[1][word], quarter, scales(pairs, c, 0), biases(pairs, c, 0), v0);
                                value_pairs<BITS>(codes[2][word], codes[3][word], quarter, scales(pairs, c, 1), biases(pairs, c, 1), v1);
#pragma unroll
                                for (int k = 0; k < 4; k += 2)
#pragma unroll
                                    for (int n = 0; n < ROWS8; ++n) {
                                        const uint32_t a[4] = {v0[k] & keep[0], v0[k + 1] & keep[0], v1[k] & keep[1], v1[k + 1] & keep[1]};
                                        float x[4];
                                        mma_f16_zc(x, a[0], a[1], a[2], a[3], pb[s][n][0], pb[s][n][1]);
                                        mma_f16(x, a[0], a[1], a[2], a[3], pl[s][n][0], pl[s][n][1]);
#pragma unroll
                                        for (int j = 0; j < 4; ++j)
                                            if (row_pos[n][j & 1] == rp) o[(c * kEach + e + k) / 2][n][j] += x[j] * (1.0f / Cfg::kUnit);
                                    }
                            }
                        }
                    }
                }
            }
            slot_done();
        }

        // join the warps: their outputs are brought to the rows' common maxima, and then only add up
        float scale[ROWS8][2];
#pragma unroll
        for (int n = 0; n < ROWS8; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float sum = l[n][j];
                m[n][j] *= unit[n][j];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
                if (gid == 0) *reinterpret_cast<float2*>(s_ml + (warp * kRows + n * 8 + quad * 2 + j) * 2) = make_float2(m[n][j], sum);
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)   // four of a group of 64
                        o[c][n][k + j] = fmaf(o[c][n][k + j], Cfg::kUnit, ob[c / 8][n][(c / 4 & 1) * 2 + j]);
                }
            }
        named_barrier(1, kThreads);
#pragma unroll
        for (int n = 0; n < ROWS8; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = n * 8 + quad * 2 + j;
                float2 ml[Cfg::kCompute];
                float top = -INFINITY, total = 0.0f;
#pragma unroll
                for (int w = 0; w < Cfg::kCompute; ++w) {
                    ml[w] = *reinterpret_cast<const float2*>(s_ml + (w * kRows + row) * 2);
                    top = fmaxf(top, ml[w].x);
                }
                const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int w = 0; w < Cfg::kCompute; ++w) total = fmaf(ml[w].y, exp2_approx(ml[w].x - ref), total);
                scale[n][j] = exp2_approx(m[n][j] - ref);
                if (warp == 0 && gid == 0) *reinterpret_cast<float2*>(s_total + row * 2) = make_float2(top, total);
            }
        const int cta = blockIdx.x;
        const bool cut = it.ua != 0 || it.ub != it.units;
        const int c0 = cut ? cta_of(it.g0, share.total, share.ctas) : cta;
        const Parts parts{p.part, p.part_ml, kRows, c0};
        // as many columns at a time as the rows leave room for; four of them at place c ^ (row / 2 % 4): no bank conflicts
        int wide = Cfg::kJoinCols;   // a power of two
        while (wide < D && 2 * wide * rows * Cfg::kCompute * 4 <= Cfg::kJoinBytes) wide *= 2;
        const int per_row = wide / 4, row_shift = 31 - __clz(per_row);
#pragma unroll 1
        for (int col0 = 0; col0 < D; col0 += wide) {
            if (col0 > 0) named_barrier(1, kThreads);
#pragma unroll
            for (int c = 0; c < kSets; ++c) {
                const int col = (c * 8 + gid) * kEach - col0;   // the lane's first
                if (col < 0 || col >= wide) continue;
#pragma unroll
                for (int n = 0; n < ROWS8; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int row = n * 8 + quad * 2 + j;
                        if (row >= rows) continue;
                        float* const at = s_join + (warp * rows + row) * wide;
#pragma unroll
                        for (int k = 0; k < kEach / 4; ++k) {
                            const float(&a)[4] = o[c * (kEach / 2) + 2 * k][n];
                            const float(&b)[4] = o[c * (kEach / 2) + 2 * k + 1][n];
                            const float by = scale[n][j];
                            *reinterpret_cast<float4*>(at + ((col / 4 + k) ^ ((row >> 1) & 3)) * 4) =
                                make_float4(a[j] * by, a[2 + j] * by, b[j] * by, b[2 + j] * by);
                        }
                    }
            }
            named_barrier(1, kThreads);
            for (int e = threadIdx.x; e < rows * per_row; e += kThreads) {
                const int row = e >> row_shift, c4 = e & (per_row - 1), d = col0 + c4 * 4;
                const float* const from = s_join + row * wide + (c4 ^ ((row >> 1) & 3)) * 4;
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < Cfg::kCompute; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(from + w * rows * wide);
                    acc.x += v.x;
                    acc.y += v.y;
                    acc.z += v.z;
                    acc.w += v.w;
                }
                const float2 total = *reinterpret_cast<const float2*>(s_total + row * 2);
                if (!cut) {
                    const float inv = total.y == 0.0f ? 0.0f : 1.0f / total.y;
                    *reinterpret_cast<uint2*>(p.out + row_offset(row, p.out_stride) + d) =
                        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                } else {
                    const int64_t at = parts.row(cta - c0, row);
                    *reinterpret_cast<float4*>(p.part + at * D + d) = acc;
                    if (d == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = total;
                }
            }
        }
        named_barrier(1, kThreads);   // the join's buffers are free for the next item
    }

    named_barrier(2, Cfg::kThreads);   // the copying warps see to the joins
}

template <int D, int BITS>
cudaError_t configure_codes_dim() {
    cudaError_t e = configure<CodesCfg<D, 1, BITS>>(qmm_attention_codes_kernel<D, 1, BITS>);
    if (e == cudaSuccess) e = configure<CodesCfg<D, 2, BITS>>(qmm_attention_codes_kernel<D, 2, BITS>);
    if (e == cudaSuccess) e = configure_tiles<D, 2, BITS>();
    if (e == cudaSuccess) e = configure_tiles<D, 4, BITS>();
    return e;
}

template <int D, int BITS>
cudaError_t launch_codes_dim(const AttnParams& p, int num_sms, cudaStream_t stream) {
    const int rows = p.rows * p.group;
    if (rows <= 8) return launch<CodesCfg<D, 1, BITS>>(qmm_attention_codes_kernel<D, 1, BITS>, p, num_sms, stream);
    if (rows <= 16) return launch<CodesCfg<D, 2, BITS>>(qmm_attention_codes_kernel<D, 2, BITS>, p, num_sms, stream);
    return rows <= 32 ? launch_tiles<D, 2, BITS>(p, num_sms, stream) : launch_tiles<D, 4, BITS>(p, num_sms, stream);
}

template <int BITS>
cudaError_t configure_codes() {
    cudaError_t e = configure_codes_dim<64, BITS>();
    if (e == cudaSuccess) e = configure_codes_dim<128, BITS>();
    if (e == cudaSuccess) e = configure_codes_dim<256, BITS>();
    return e;
}

template <int BITS>
cudaError_t launch_codes(int head_dim, const AttnParams& p, int num_sms, cudaStream_t stream) {
    if (head_dim == 64) return launch_codes_dim<64, BITS>(p, num_sms, stream);
    if (head_dim == 128) return launch_codes_dim<128, BITS>(p, num_sms, stream);
    return launch_codes_dim<256, BITS>(p, num_sms, stream);
}

}  // namespace

}  // namespace qmmk
