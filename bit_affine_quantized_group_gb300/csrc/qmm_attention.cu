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
#include "qmm_attention_tiles.cuh"

#include <atomic>

namespace qmmk {

namespace {

template <int D>
cudaError_t configure_dim() {
    cudaError_t e = configure_tiles<D, 1, 16>();
    if (e == cudaSuccess) e = configure_tiles<D, 2, 16>();
    if (e == cudaSuccess) e = configure_tiles<D, 4, 16>();
    return e;
}

template <int D>
cudaError_t launch_dim(const AttnParams& p, int num_sms, cudaStream_t stream) {
    const int rw = attn_row_warps(p.rows * p.group);
    if (rw == 1) return launch_tiles<D, 1, 16>(p, num_sms, stream);
    return rw == 2 ? launch_tiles<D, 2, 16>(p, num_sms, stream) : launch_tiles<D, 4, 16>(p, num_sms, stream);
}

}  // namespace

cudaError_t configure_attention() {
    cudaError_t e = configure_dim<64>();
    if (e == cudaSuccess) e = configure_dim<128>();
    if (e == cudaSuccess) e = configure_dim<256>();
    return e;
}

// Once for each device and kind of codes, by the first call: a plan does not know its calls' caches, and what is configured is
// loaded.
cudaError_t configure_attention_codes(int bits, int device) {
    static std::atomic<uint64_t> done[2];   // of 8 and of 4 bits: one bit for each device
    std::atomic<uint64_t>& of = done[bits == 8 ? 0 : 1];
    if (device < 64 && of.load(std::memory_order_acquire) >> device & 1) return cudaSuccess;
    const cudaError_t e = bits == 8 ? configure_attention_codes8() : configure_attention_codes4();
    if (e == cudaSuccess && device < 64) of.fetch_or(1ull << device, std::memory_order_release);
    return e;
}

cudaError_t launch_attention(int head_dim, int bits, const AttnParams& p, int num_sms, cudaStream_t stream) {
    if (bits == 8) return launch_attention_codes8(head_dim, p, num_sms, stream);
    if (bits == 4) return launch_attention_codes4(head_dim, p, num_sms, stream);
    if (head_dim == 64) return launch_dim<64>(p, num_sms, stream);
    if (head_dim == 128) return launch_dim<128>(p, num_sms, stream);
    return launch_dim<256>(p, num_sms, stream);
}

}  // namespace qmmk
