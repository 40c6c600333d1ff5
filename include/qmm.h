/*
 * qmm.h -- C ABI of the GB300 (sm_103a) group-wise affine-quantized
 * multi-row matmul.
 *
 * The operation (vmlx-swift PR #565 "Enable bundle-aware Qwen speculation and
 * dense mixed JANGH loading", LaneQMM commit: matmul over raw affine codes with
 * the dequant applied after the dot product, "C += s*P + b*XS"):
 *
 *   y[m,n] = sum_g ( s[n,g] * P[m,n,g] + b[n,g] * XS[m,g] )
 *   P[m,n,g] = sum_{k in g} x[m,k] * q[n,k]      XS[m,g] = sum_{k in g} x[m,k]
 *
 * which equals x . W^T with W[n,k] = s[n,k/group] * q[n,k] + b[n,k/group].
 * It serves decode (M = 1) and speculative-decoding verification (M = 2..16
 * rows; same page, LaneQMM and qwen_qmv_rows_full commits: weight words, scales
 * and biases are read once for all rows).
 *
 * Data layout (all row-major, all owned by the caller):
 *   x       [M, K]          bfloat16 activations
 *   w       [N, K*bits/32]  uint32 words; row n holds q[n, 0..K-1] as an
 *                           LSB-first bit stream: bit j of code k is bit
 *                           (k*bits + j) mod 32 of word (k*bits + j) / 32.
 *                           5- and 6-bit codes may straddle two words.
 *   scales  [N, K/group]    IEEE binary16
 *   biases  [N, K/group]    IEEE binary16
 *   out     [M, N]          float32 or bfloat16 (round to nearest even),
 *                           overwritten (never accumulated into).
 *
 * Supported formats: bits in {2, 3, 4, 5, 6, 8}, group in {32, 64}, 1 <= M <= 16.
 * (2-bit tensors are in use beside 4/8-bit ones per "Qwen3.8 Flash Next
 * performance and parity receipt", MTPLX logic review, and the "JANGH split-K
 * verify tile" commit tests 2/4/8-bit codes; 3-bit follows the same stream.)
 * Requirements checked before any launch: K % group == 0; K*bits % 128 == 0
 * (every packed row starts on a 16-byte boundary); K/group even (so K is a
 * multiple of 64); x, packed weights, scales and biases 16-byte aligned
 * device pointers (x is read with tensor-memory-access copies); out a
 * naturally aligned device pointer.
 *
 * Split-K (same page, commit "JANGH split-K verify tile": K is sliced across
 * the grid, FP32 partials are written and then summed): with splits S > 1 the
 * K range is cut into S slices on 8-group chunk boundaries (uneven slices
 * allowed), each slice writes float32 partials into the plan's workspace and a
 * second kernel sums them in slice order 0..S-1, so results are deterministic
 * run to run but not bitwise equal to S = 1 (the page's contract: not
 * bitwise, covered by tolerance tests).
 *
 * Banked mode (same page, qwen_qmv_rows_full commit: 36 projection banks in
 * one dispatch) runs several projections that share x in one launch.
 *
 * Conventions:
 *   - Every function returns a qmm_status (0 = QMM_OK) and never throws.
 *   - qmm_forward / qmm_forward_banked / qmm_forward_swiglu are asynchronous on `stream` (a
 *     cudaStream_t passed as void*, NULL = legacy default stream); they never
 *     allocate and never synchronize. Errors in arguments are reported before
 *     anything is launched. Launch failures return QMM_ERR_CUDA.
 *   - A plan (and its workspace) must be used by one stream at a time.
 *   - All device pointers must stay valid until the stream work completes.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
enum {
    QMM_OK = 0,
    QMM_ERR_INVALID_ARG = 1,   /* NULL/misaligned pointer, out-of-range value */
    QMM_ERR_UNSUPPORTED = 2,   /* well-formed request this library does not implement */
    QMM_ERR_PLAN_MISMATCH = 3, /* K/N/bits/group differ from the plan's */
    QMM_ERR_CUDA = 4,          /* a CUDA runtime call failed (no device, launch error) */
    QMM_ERR_ALLOC = 5,         /* host or device allocation failed in qmm_plan */
    QMM_ERR_TIMEOUT = 6,       /* a kernel gave up a bounded wait (qmm_plan_error) */
    QMM_ERR_SCRATCH_LIMIT = 7  /* reserved (no longer returned: qmm_forward_noalloc lowers its K slices to fit) */
};

/* Output element types. */
enum { QMM_OUT_F32 = 0, QMM_OUT_BF16 = 1 };

#define QMM_MAX_ROWS 16
#define QMM_MAX_BANKS 64
#define QMM_MAX_SPLITS 16

/* Problem descriptor fixed at plan time. */
typedef struct qmm_desc {
    int64_t K;          /* reduction length (codes per weight row) */
    int64_t N;          /* output columns (weight rows) */
    int32_t bits;       /* code width: 2, 3, 4, 5, 6 or 8 */
    int32_t group;      /* codes per scale/bias group: 32 or 64 */
    int32_t max_M;      /* largest M forward will be called with, 1..16 */
    int32_t out_dtype;  /* QMM_OUT_F32 or QMM_OUT_BF16 */
    int32_t splits;     /* 0 = choose automatically, else 1..16 K slices */
    int32_t max_banks;  /* largest n_banks for qmm_forward_banked, 1..64 */
} qmm_desc;

/* What a plan decided (for reporting and tests). */
typedef struct qmm_plan_info {
    int32_t splits;          /* K slices used by every forward call */
    int32_t chunks;          /* 8-group chunks along K */
    int32_t stages[2];       /* weight-pipeline depth of the main kernel a single-projection call
                                of M <= 8 rows uses, and of the one for 9 <= M <= 16 */
    int32_t smem_bytes[2];   /* dynamic shared memory per CTA, same order */
    int32_t num_sms;         /* streaming multiprocessors on the plan's device */
    int32_t device;          /* CUDA device ordinal the plan was made on */
    int64_t workspace_bytes; /* device workspace the plan uses */
} qmm_plan_info;

typedef struct qmm_plan qmm_plan_t;

/*
 * Validate a descriptor on the host (no CUDA call). Returns QMM_OK,
 * QMM_ERR_INVALID_ARG (malformed: NULL, K % group != 0, out-of-range
 * max_M/out_dtype/splits/max_banks) or QMM_ERR_UNSUPPORTED (well formed but
 * outside this library: other bit widths or group sizes, K*bits % 128 != 0,
 * K/group odd, splits greater than the number of 8-group chunks).
 */
int qmm_validate_desc(const qmm_desc* d);

/*
 * Device workspace a plan for `d` needs (bytes; 0 if d is invalid): a
 * 256-byte error word plus split-K partials for max_banks * splits * max_M * N
 * floats (splits = 0 is sized for the largest automatic choice,
 * min(8, chunks) with chunks = ceil(K / group / 8)). Lets the caller
 * (e.g. PyTorch's allocator) own it.
 */
size_t qmm_workspace_bytes(const qmm_desc* d);

/*
 * Create a plan on the current CUDA device. Validates `d`, queries the device
 * (SM count, shared memory), picks splits when d->splits == 0, and configures
 * the kernels. If `workspace` is NULL the plan cudaMallocs its own workspace of
 * qmm_workspace_bytes(d) bytes (freed by qmm_destroy); otherwise `workspace`
 * must be a device pointer, 256-byte aligned, of at least ws_bytes >=
 * qmm_workspace_bytes(d) bytes, owned by the caller and not used by anything
 * else while the plan is in use. Its error word is cleared on the legacy
 * default stream before the call returns, so nothing launched before, on any
 * stream, may write the workspace any more. On failure *plan is set to NULL.
 */
int qmm_plan(qmm_plan_t** plan, const qmm_desc* d, void* workspace, size_t ws_bytes);

/* Copy out what the plan decided. */
int qmm_plan_get_info(const qmm_plan_t* p, qmm_plan_info* info);

/*
 * Host-only check of forward arguments against a descriptor, exactly as
 * qmm_forward_banked performs it before launching (n_banks arrays of device
 * pointers; qmm_forward is the n_banks == 1 case). No CUDA call. Returns
 * QMM_OK, QMM_ERR_INVALID_ARG (NULL or misaligned pointer, M < 0,
 * M > max_M, n_banks out of range) or QMM_ERR_PLAN_MISMATCH.
 */
int qmm_check_forward_args(const qmm_desc* d, const void* x_bf16, int M, int n_banks,
                           const uint32_t* const* packed_w, const uint16_t* const* scales_f16,
                           const uint16_t* const* biases_f16, int64_t K, int64_t N, int bits,
                           int group, void* const* out);

/*
 * y = qmm(x, w, scales, biases) for one projection. M = 0 is a no-op that
 * returns QMM_OK. K, N, bits and group must equal the plan's
 * (QMM_ERR_PLAN_MISMATCH otherwise); M must be <= the plan's max_M.
 * Launches, in stream order: the main kernel (it streams the weights, stages
 * the activations and computes the projection) and, when the plan's
 * splits > 1, the split-K reduce kernel.
 *
 * Ordering: x is read only after the work issued before the call on the
 * stream has finished, and out is written after that too. The packed weights,
 * scales and biases are streamed from the start (programmatic dependent
 * launch), possibly while that earlier work still runs: they must not be
 * written by work issued just before the call (weights are normally written
 * once, at load time; synchronize the stream or record/wait an event in
 * between otherwise). The same holds for every forward entry point.
 */
int qmm_forward(const qmm_plan_t* p, const void* x_bf16, int M, const uint32_t* packed_w,
                const uint16_t* scales_f16, const uint16_t* biases_f16, int64_t K, int64_t N,
                int bits, int group, void* out, void* stream);

/*
 * n_banks projections of the same shape and format that share x, in one
 * launch of the main kernel. packed_w, scales_f16, biases_f16 and out are HOST
 * arrays of n_banks device pointers (copied into the kernel parameters; the
 * arrays may be reused as soon as the call returns). 1 <= n_banks <= the
 * plan's max_banks (<= 64). Each bank's result equals qmm_forward on that bank
 * with the same plan.
 */
int qmm_forward_banked(const qmm_plan_t* p, const void* x_bf16, int M, int n_banks,
                       const uint32_t* const* packed_w, const uint16_t* const* scales_f16,
                       const uint16_t* const* biases_f16, int64_t K, int64_t N, int bits,
                       int group, void* const* out, void* stream);

/*
 * Fused gate/up projection with a SwiGLU epilogue ("Qwen3.8 Flash Next
 * performance and parity receipt": the exact fused projection promoted over
 * separate gate and up projections):
 *   out[m, n] = silu(gate[m, n]) * up[m, n],   silu(g) = g / (1 + exp(-g)),
 * where gate and up are the qmm_forward results of (w_gate, s_gate, b_gate)
 * and (w_up, s_up, b_up) on the same x, both N x K in the plan's format. One
 * launch of the main kernel computes both: every CTA runs each of its row
 * blocks for the gate and then for the up weights, keeping the fp32 gate
 * values in the plan's workspace. The plan must have max_banks >= 2 (else
 * QMM_ERR_INVALID_ARG). With splits > 1 both projections write fp32 slice
 * partials and the reduce kernel applies the epilogue to the slice sums.
 * Pointers and argument checks as for qmm_forward; out is [M, N] in the
 * plan's output type.
 */
int qmm_forward_swiglu(const qmm_plan_t* p, const void* x_bf16, int M, const uint32_t* w_gate,
                       const uint16_t* s_gate, const uint16_t* b_gate, const uint32_t* w_up,
                       const uint16_t* s_up, const uint16_t* b_up, int64_t K, int64_t N, int bits,
                       int group, void* out, void* stream);

/*
 * Diagnostic: run the main kernel's in-register code unpacking on packed
 * weights and write the decoded codes, codes[n*K + k] = q[n,k] (uint8, device
 * pointer, N*K bytes). A code whose unpacked binary16 image is not the exact
 * value 1024 + q * 2^j (j the code's mantissa shift) is written as 0xFF.
 * Asynchronous on `stream`.
 */
int qmm_unpack_codes(const uint32_t* packed_w, int64_t K, int64_t N, int bits, uint8_t* codes,
                     void* stream);

/*
 * Wait for the device, then read and clear the plan's device error word, which
 * is done when the call returns (no call of the plan may be made meanwhile).
 * Sets *flags to 0 when every kernel since the last call finished normally; nonzero when a
 * kernel gave up a bounded wait (its output is then incomplete) and returns
 * QMM_ERR_TIMEOUT in that case.
 */
int qmm_plan_error(const qmm_plan_t* p, uint32_t* flags);

/*
 * Size of the device scratch qmm_forward_noalloc keeps in a static device
 * array (held by every GPU that loads this library until the process exits).
 */
#define QMM_NOALLOC_SCRATCH_BYTES (4u << 20)

/*
 * qmm_forward without a plan and without any allocation, for callers that
 * cannot call cudaMalloc when they run a projection (code that runs while
 * another component owns the device allocator, loops that forbid allocation
 * after start-up, plug-in hosts that only hand over their tensors). The pages
 * describe no counterpart: this is a deployment variant of qmm_forward.
 *
 * Same arguments, data layout and kernels as qmm_forward, with the output
 * type given directly (QMM_OUT_F32 or QMM_OUT_BF16). The device scratch that
 * qmm_forward keeps in its plan's workspace (the kernels' error word and the
 * fp32 partial sums of K slices) lives in a static device array of
 * QMM_NOALLOC_SCRATCH_BYTES. The K-slice count is the one an automatic plan
 * would choose, lowered until 256 + slices * M * N * 4 bytes fit the array
 * (one slice needs no partials), so every supported shape runs; results are
 * bitwise those of qmm_forward with a plan of that slice count. Nothing is
 * allocated: no cudaMalloc, no cudaFree, no allocating library routine.
 *
 * The first call on a device (with that device current) looks up the
 * scratch's device address and sets the kernels' shared-memory limit; make
 * that first call before any stream capture. Every call on a device shares the
 * one scratch array and overwrites it, so calls whose executions overlap on
 * the GPU (different streams, or concurrent host threads) race: serialize
 * them. Device-side timeouts are recorded only in the scratch and not
 * reported; use qmm_forward for that.
 */
int qmm_forward_noalloc(const void* x_bf16, int M, const uint32_t* packed_w, const uint16_t* scales_f16,
                        const uint16_t* biases_f16, int64_t K, int64_t N, int bits, int group, int out_dtype,
                        void* out, void* stream);

/* Free the plan and any workspace it allocated. NULL is accepted. */
void qmm_destroy(qmm_plan_t* p);

/*
 * ---------------------------------------------------------------------------
 * Between two projections of a decode or verification step: query/key norms
 * with the position rotation and the append to a paged key/value cache,
 * attention of the new tokens over that cache, and the draw of the next token
 * from the output head's logits.
 *
 * A step has `seqs` sequences of `rows` new tokens each; token t = s * rows + r
 * is row r of sequence s. lengths[s] (device int32) counts the tokens of
 * sequence s with the new ones, so row r has the cache position
 *   pos(s, r) = lengths[s] - rows + r.
 * A row with pos < 0 is padding: nothing is appended for it, and it attends to
 * nothing (its output is zeros).
 *
 * The cache is a pool of pages of page_size positions. Position j of sequence s
 * is slot j % page_size of page page_table[s * max_pages + j / page_size]
 * (device int32). Entries of positions that no row reads or writes are never
 * used and may hold anything. Elements are bfloat16 at
 *   base + page * page_stride + head * head_stride + slot * slot_stride + d.
 */

#define QMM_KV_MAX_SEQS 65536
#define QMM_KV_MAX_ROWS 16
#define QMM_KV_MAX_GROUP 64

/* Types of the values that qmm_qk_norm_rope and qmm_sample read. */
enum { QMM_IN_F32 = 0, QMM_IN_BF16 = 1 };

/* Error bits of qmm_kv_error. */
enum {
    QMM_KV_TIMEOUT = 7,       /* a kernel gave up a bounded wait (any of three bits) */
    QMM_KV_BAD_PAGE = 16,     /* a page table entry in use lies outside 0..num_pages-1: read as zeros, not written */
    QMM_KV_BAD_LENGTH = 32,   /* a length above max_pages * page_size: rows stand where it says, and what is past the page
                                 table was neither written nor seen */
    QMM_KV_BAD_POSITION = 64, /* a rotation position outside the rope table: the row was not rotated */
    QMM_KV_NOT_FINITE = 128   /* an infinity or NaN was appended to a cache of codes */
};

/* What a plan for the cache operators fixes. */
typedef struct qmm_kv_desc {
    int32_t q_heads;      /* query heads, a multiple of kv_heads (at most QMM_KV_MAX_GROUP times as many) */
    int32_t kv_heads;     /* heads of the cache */
    int32_t head_dim;     /* 64, 128 or 256 */
    int32_t page_size;    /* positions of a page: a power of two, 1..1024 */
    int32_t max_seqs;     /* largest number of sequences of a call */
    int32_t max_rows;     /* largest rows of an attention call, 1..16 */
    int32_t max_pages;    /* entries of a page table row (the table is [seqs, max_pages]) */
    int32_t window;       /* 0: every earlier position is visible; W: those with pos - j < W ... */
    int32_t sinks;        /* ... and the first `sinks` positions */
    int32_t rot_dim;      /* rotated elements of a head: 0 or a multiple of 16, at most head_dim */
    int32_t interleaved;  /* 0: element i turns with i + rot_dim/2; 1: element 2i with 2i + 1 */
    float scale;          /* factor of the attention scores */
    float eps;            /* added to the mean square in the norms */
} qmm_kv_desc;

/* The cache: bases, pages, and strides in elements (multiples of 8). */
typedef struct qmm_kv_cache {
    void* k;              /* bfloat16, 16-byte aligned */
    void* v;
    int64_t num_pages;
    int64_t k_page_stride, k_head_stride, k_slot_stride;
    int64_t v_page_stride, v_head_stride, v_slot_stride;
} qmm_kv_cache;

typedef struct qmm_kv_plan qmm_kv_plan_t;

/* Validate a descriptor on the host (no CUDA call): QMM_OK, QMM_ERR_INVALID_ARG or QMM_ERR_UNSUPPORTED. */
int qmm_kv_validate_desc(const qmm_kv_desc* d);

/* Device workspace of a plan for `d` (error word, join counters and partial results); 0 if d is invalid. */
size_t qmm_kv_workspace_bytes(const qmm_kv_desc* d);

/*
 * Create a plan on the current device, where its calls run whatever device is
 * current then; the workspace is handled as in qmm_plan (NULL: the plan
 * allocates it). Its head is cleared on the legacy default stream before the
 * call returns, so nothing launched before, on any stream, may write the
 * workspace any more. A plan is used by one stream at a time; qmm_qk_norm_rope
 * and qmm_attention may share one, and so may host threads that launch on the
 * same stream.
 */
int qmm_kv_plan(qmm_kv_plan_t** plan, const qmm_kv_desc* d, void* workspace, size_t ws_bytes);

/*
 * Wait for the device, then read and clear the plan's error word, which is
 * done when the call returns: QMM_ERR_TIMEOUT or QMM_ERR_INVALID_ARG if a bit
 * was set. No call of the plan may be made meanwhile.
 */
int qmm_kv_error(const qmm_kv_plan_t* p, uint32_t* flags);

/* Free the plan and any workspace it allocated. NULL is accepted. */
void qmm_kv_destroy(qmm_kv_plan_t* p);

/* What qmm_qk_norm_rope reads and writes. All pointers are device pointers. */
typedef struct qmm_append_args {
    const void* q;            /* [seqs*rows, q_heads*head_dim], in_dtype, 16-byte aligned rows */
    const void* k;            /* [seqs*rows, kv_heads*head_dim] */
    const void* v;            /* [seqs*rows, kv_heads*head_dim] */
    int64_t q_stride, k_stride, v_stride;   /* elements from row to row (multiples of 16 bytes) */
    const float* q_weight;    /* [head_dim] norm weights, 16-byte aligned; NULL: queries are not normalised */
    const float* k_weight;    /* [head_dim]; NULL: keys are not normalised */
    const float* rope;        /* [rope_len, rot_dim]: rot_dim/2 cosines, then rot_dim/2 sines; 16-byte aligned */
    int64_t rope_len;
    const int32_t* lengths;   /* [seqs] */
    const int32_t* positions; /* [seqs*rows] rotation positions; NULL: the cache positions */
    const int32_t* page_table;/* [seqs, max_pages] */
    void* q_out;              /* [seqs*rows, q_heads*head_dim] bfloat16, 16-byte aligned rows */
    int64_t q_out_stride;
    int32_t seqs;             /* <= max_seqs */
    int32_t rows;             /* any number: prompts too */
    int32_t in_dtype;         /* QMM_IN_F32 or QMM_IN_BF16 (a projection's output type) */
} qmm_append_args;

/*
 * For every new token and head: y = x * rsqrt(mean(x^2) + eps) * weight for
 * queries and keys, the first rot_dim elements rotated by the token's position,
 * all in float32, rounded once to bfloat16; queries go to q_out, keys and the
 * (only rounded) values to their cache slots. One launch. q_out rows of padding
 * are zeros. q_out must not overlap the inputs.
 * The host-only check makes no CUDA call.
 */
int qmm_check_qk_norm_rope_args(const qmm_kv_desc* d, const qmm_kv_cache* cache, const qmm_append_args* a);
int qmm_qk_norm_rope(const qmm_kv_plan_t* p, const qmm_kv_cache* cache, const qmm_append_args* a, void* stream);

/* What qmm_attention reads and writes. All pointers are device pointers. */
typedef struct qmm_attention_args {
    const void* q;             /* [seqs*rows, q_heads*head_dim] bfloat16, 16-byte aligned rows */
    void* out;                 /* as q */
    const int32_t* lengths;    /* [seqs] */
    const int32_t* page_table; /* [seqs, max_pages] */
    int64_t q_stride, out_stride;   /* elements from row to row (multiples of 16 bytes) */
    int32_t seqs;              /* <= max_seqs */
    int32_t rows;              /* <= max_rows */
} qmm_attention_args;

/*
 * out[t, h] = sum_j softmax_j(scale * q[t, h] . k_j) v_j over the positions j
 * that token t sees: j <= pos, and with a window pos - j < window or j < sinks.
 * Query head h reads cache head h / (q_heads / kv_heads). The scores, the
 * softmax's maximum and sum and the output are held in float32, the output
 * until its end as the sum before the division: values from 2^127 / positions
 * on can overflow it. A row that sees nothing gives zeros, and no value at a
 * position that a row does not see reaches that row, infinities and NaN among
 * them.
 *
 * The work of all sequences is cut into equal shares for the GPU whatever their
 * lengths; the parts of one head are joined in a fixed order, so a call with
 * the same lengths gives the same bits. The cut depends on all lengths of the
 * call: the same sequence in another batch may differ by rounding.
 */
int qmm_check_attention_args(const qmm_kv_desc* d, const qmm_kv_cache* cache, const qmm_attention_args* a);
int qmm_attention(const qmm_kv_plan_t* p, const qmm_kv_cache* cache, const qmm_attention_args* a, void* stream);

/*
 * ---------------------------------------------------------------------------
 * The same operators over a cache of codes: every 64 elements of a head
 * (positions are quantised one by one) are held as 8- or 4-bit codes c with a
 * binary16 scale s and bias b, and stand for s c + b, as a projection's weights
 * do. Code j of a head lies in bits j * bits .. j * bits + bits - 1 of its bytes
 * (4 bits: the even code in the low half).
 *
 * Values x are quantised in float32, after norm and rotation and without a
 * rounding before:
 *   lo, hi = least and largest of the 64,   b = f16(lo),   s = f16((hi - lo) / top),
 *   c = round((x - b) * (1 / s)) brought to 0..top,   c = 0 where s = 0,
 * with top = 255 or 15, and roundings to the nearest, ties to even. An element
 * is held within s/2 + 2^-11 (|lo| + |hi|) + 2^-17, times 1 + 2^-10. Elements
 * beyond +-QMM_KVQ_LARGEST are brought to it and NaN to 0, so that what is
 * appended is always finite; an infinity or NaN among them sets
 * QMM_KV_NOT_FINITE in the plan's error word.
 */
#define QMM_KVQ_GROUP 64
#define QMM_KVQ_LARGEST 65280

/* The cache: as qmm_kv_cache, with strides of the codes in bytes (multiples of 16) and of the scales and biases in
   pairs (multiples of head_dim / 64). */
typedef struct qmm_kvq_cache {
    void* k;              /* codes, head_dim * bits / 8 bytes of a head, 16-byte aligned */
    void* v;
    void* k_affine;       /* (scale, bias) binary16 pairs, head_dim / 64 of a head, 16-byte aligned */
    void* v_affine;
    int64_t num_pages;
    int64_t k_page_stride, k_head_stride, k_slot_stride;
    int64_t v_page_stride, v_head_stride, v_slot_stride;
    int64_t ka_page_stride, ka_head_stride, ka_slot_stride;
    int64_t va_page_stride, va_head_stride, va_slot_stride;
    int32_t bits;         /* 8 or 4 */
} qmm_kvq_cache;

/* qmm_qk_norm_rope with keys and values quantised as they are written. The same plan, arguments and checks. */
int qmm_check_kvq_qk_norm_rope_args(const qmm_kv_desc* d, const qmm_kvq_cache* cache, const qmm_append_args* a);
int qmm_kvq_qk_norm_rope(const qmm_kv_plan_t* p, const qmm_kvq_cache* cache, const qmm_append_args* a, void* stream);

/*
 * qmm_attention over a cache of codes. The same plan, arguments and checks. Each
 * query row enters as binary16 numbers of a power of two that brings its largest
 * element to 2^14..2^15 (elements down to 2^-28 of that keep all bits). Scores are
 * products with the codes themselves, scaled in float32. Where rows * q_heads /
 * kv_heads is up to 16, the values' scales enter with the softmax's weights, which
 * are two binary16 terms. With P a position's weight relative to the row's largest (or
 * the largest among 32 neighbours, where that is more) and top 255 or 15, its share of
 * an output is off by up to (2^-19 P + 2^-37) (|s| top + |b|) + 2^-30.
 * Of more, values enter as binary16, s c + b rounded once (within 2^-11 of it or 2^-25),
 * and weights within 2^-11 or, of the largest, 2^-40; so do values of 32 neighbouring
 * positions where an |s| is 2 or more (8 for 4 bits). Sums and maxima are float32.
 * s c + b beyond binary16 may be infinite.
 */
int qmm_check_kvq_attention_args(const qmm_kv_desc* d, const qmm_kvq_cache* cache, const qmm_attention_args* a);
int qmm_kvq_attention(const qmm_kv_plan_t* p, const qmm_kvq_cache* cache, const qmm_attention_args* a, void* stream);

/* What qmm_kvq_read reads and writes. All pointers are device pointers. */
typedef struct qmm_read_args {
    void* k_out;               /* row j of sequence s at k_out + s * k_seq_stride + j * k_row_stride: kv_heads * head_dim */
    void* v_out;               /* elements of out_dtype, 16-byte aligned rows */
    int64_t k_seq_stride, k_row_stride;   /* elements (multiples of 16 bytes) */
    int64_t v_seq_stride, v_row_stride;
    const int32_t* lengths;    /* [seqs] */
    const int32_t* starts;     /* [seqs] the position of row 0; NULL: 0 */
    const int32_t* page_table; /* [seqs, max_pages] */
    int32_t seqs;              /* <= max_seqs */
    int32_t rows;              /* rows of k_out and v_out for a sequence */
    int32_t out_dtype;         /* QMM_OUT_F32 or QMM_OUT_BF16 */
} qmm_read_args;

/*
 * Reads a cache of codes back: row j of sequence s gets s c + b of position
 * starts[s] + j, exact in float32 but for one rounding, for positions from 0 to
 * lengths[s] - 1. Rows of other positions are left as they were. Pages and
 * lengths that are out of range are treated as in qmm_attention (zeros, and a
 * bit of the error word). k_out, v_out and the cache do not overlap. One launch.
 */
int qmm_check_kvq_read_args(const qmm_kv_desc* d, const qmm_kvq_cache* cache, const qmm_read_args* a);
int qmm_kvq_read(const qmm_kv_plan_t* p, const qmm_kvq_cache* cache, const qmm_read_args* a, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a projection that they share:
 *   out[m, :] = y[m, :] + scale[i] * (x[m, :] . A[i]^T) . B[i]^T,   i = ids[m],
 * with y the projection's result for x. A row with id -1 has none: out = y.
 * Rows of an adapter may stand anywhere. Adapters of a smaller rank are filled
 * up with zero rows of A (and zero columns of B).
 */
#define QMM_ADAPTER_MAX_RANK 128
#define QMM_ADAPTER_MAX_ROWS (1 << 20)

enum { QMM_ADAPTER_BAD_ID = 1 };   /* error bit: an id outside -1..adapters-1, treated as -1 */

/* What a plan for adapters fixes. */
typedef struct qmm_adapter_desc {
    int64_t K;          /* width of x, a multiple of 64 */
    int64_t N;          /* width of y and out */
    int32_t rank;       /* a multiple of 8, at most QMM_ADAPTER_MAX_RANK */
    int32_t adapters;   /* how many A and B hold */
    int32_t max_rows;   /* largest rows of a call, at most QMM_ADAPTER_MAX_ROWS */
    int32_t out_dtype;  /* of y and out: QMM_OUT_F32 or QMM_OUT_BF16 */
} qmm_adapter_desc;

typedef struct qmm_adapter_plan qmm_adapter_plan_t;

/* Validate a descriptor on the host (no CUDA call): QMM_OK, QMM_ERR_INVALID_ARG or QMM_ERR_UNSUPPORTED. */
int qmm_adapter_validate_desc(const qmm_adapter_desc* d);

/* Device workspace of a plan for `d` (error word and x . A^T of max_rows rows); 0 if d is invalid. */
size_t qmm_adapter_workspace_bytes(const qmm_adapter_desc* d);

/* Create a plan on the current device; device, workspace, streams and threads as for qmm_kv_plan. */
int qmm_adapter_plan(qmm_adapter_plan_t** plan, const qmm_adapter_desc* d, void* workspace, size_t ws_bytes);

/* Wait for the device, then read and clear the plan's error word, as qmm_kv_error. */
int qmm_adapter_error(const qmm_adapter_plan_t* p, uint32_t* flags);

/* Free the plan and any workspace it allocated. NULL is accepted. */
void qmm_adapter_destroy(qmm_adapter_plan_t* p);

/* What qmm_add_adapters reads and writes. All pointers are device pointers. */
typedef struct qmm_adapter_args {
    const void* x;        /* [rows, K] bfloat16, 16-byte aligned rows */
    const void* a;        /* [adapters, rank, K] bfloat16, 16-byte aligned */
    const void* b;        /* [adapters, N, rank] bfloat16, 16-byte aligned */
    const float* scale;   /* [adapters]; NULL: 1 */
    const int32_t* ids;   /* [rows] */
    const void* y;        /* [rows, N] of out_dtype; may be out */
    void* out;            /* [rows, N] */
    int64_t x_stride;     /* elements from row to row (a multiple of 8) */
    int64_t y_stride, out_stride;
    int32_t rows;
} qmm_adapter_args;

/*
 * Adds the adapters' products. x . A^T is summed in float32 and enters the
 * second product as bfloat16 terms (two within 2^-17, for float32 outputs three
 * within 2^-26); that is summed in float32 with y and rounded once. A lower term
 * may be 0, and 0 times an infinity of B is NaN, so that an infinite element of B
 * makes its column of the adapter's rows NaN. The order of the sums is fixed: a
 * call gives the same bits for the same inputs. out may be y itself (rows at the
 * same places) and otherwise overlaps nothing. Two launches, of which the second
 * reads ids, y and b while the first still runs: they are written by nothing but
 * what came before the call on its stream (or was waited for there), and by nothing
 * while the call runs but the call itself. rows = 0 is a no-op.
 */
int qmm_check_adapter_args(const qmm_adapter_desc* d, const qmm_adapter_args* a);
int qmm_add_adapters(const qmm_adapter_plan_t* p, const qmm_adapter_args* a, void* stream);

/* Largest vocabulary of qmm_sample. */
#define QMM_SAMPLE_MAX_VOCAB 393216

/*
 * Draw one token for each of M rows of logits [M, vocab] (rows `stride`
 * elements apart; naturally aligned) from the given uniform numbers u[M].
 * With the row's temperature T, top_k, top_p and min_p (device arrays [M]):
 *   w_i = exp((l_i - max l) / T), held as the whole number floor(2^40 w_i);
 *   tokens are ranked by falling logit, equal ones by rising index, and kept if
 *     rank < top_k                      (top_k <= 0: no limit),
 *     the mass ranked before it < top_p * the mass of the top_k  (top_p >= 1: no limit),
 *     w_i >= min_p                      (min_p <= 0: no limit);
 *   the token of rank 0 is always kept;
 *   token = the first index whose sum of kept mass up to itself exceeds
 *     floor(u * kept mass), and prob = its mass / the kept mass.
 * The masses are whole numbers, so no order of summation changes a result. T
 * not above 0 takes the token of rank 0. NaN logits count as -infinity; a row
 * without any logit above that gives token -1 and prob 0. u outside [0, 1) is
 * brought to the nearest kept mass. probs may be NULL. 1 <= vocab <=
 * QMM_SAMPLE_MAX_VOCAB. M = 0 is a no-op. One launch, on the current
 * device; no plan, no workspace.
 */
int qmm_sample(const void* logits, int M, int vocab, int64_t stride, int in_dtype, const float* temperature,
               const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* tokens,
               float* probs, void* stream);

/* Most alternatives of qmm_logprobs. */
#define QMM_LOGPROBS_MAX_TOP 32

/*
 * Log probabilities of M rows of logits [M, vocab] (as for qmm_sample, rows
 * `stride` elements apart), in one pass over them: with
 *   lse = log sum_i exp(l_i),
 *   token_logprobs[m] = l_t - lse for the given token t = tokens[m],
 *   entropy[m] = -sum_i p_i log p_i, p_i = exp(l_i - lse),
 *   top_tokens[m, 0..top-1], top_logprobs[m, 0..top-1]: the tokens of the largest
 *     logits by falling logit, equal ones by rising index, and their l_i - lse.
 * NaN logits count as -infinity and +infinity as the largest float32. A token
 * outside 0..vocab-1 has the log probability -infinity; so has every token of a
 * row without any logit above -infinity, whose entropy is 0. Places past the
 * vocabulary get token -1 and -infinity. tokens and token_logprobs may both be
 * NULL, and so may entropy; top = 0 with both of its arrays NULL asks for no
 * alternatives (0 <= top <= QMM_LOGPROBS_MAX_TOP). 1 <= vocab <=
 * QMM_SAMPLE_MAX_VOCAB. M = 0 is a no-op. One launch, on the current device; no
 * plan, no workspace. The same logits give the same bits, for one number of rows
 * and one place of the row's first logit in its 16 bytes.
 */
int qmm_logprobs(const void* logits, int M, int vocab, int64_t stride, int in_dtype, const int32_t* tokens,
                 float* token_logprobs, float* entropy, int top, int32_t* top_tokens, float* top_logprobs, void* stream);

/* Static description of a status code; never NULL. */
const char* qmm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
