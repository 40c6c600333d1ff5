// C ABI of the cache operators: descriptor and argument checks, plans, and the
// calls of qmm_qk_norm_rope and qmm_attention. The contract is in include/qmm.h.
#include <cuda_runtime.h>
#include <pthread.h>

#include <cmath>
#include <cstring>
#include <new>

#include "../../include/qmm.h"
#include "qmm_kv.h"

using namespace qmmk;

struct qmm_kv_plan {
    qmm_kv_desc d;
    int device;
    int num_sms;
    uint8_t* ws;
    bool owns_ws;
    // held while an attention call launches: the kernel that joins parts reads what the one before it left in the workspace,
    // and no other thread's call may come between the two
    mutable pthread_mutex_t launches = PTHREAD_MUTEX_INITIALIZER;
};

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

int check_cache(const qmm_kv_cache* c) {
    if (c == nullptr || c->k == nullptr || c->v == nullptr) return QMM_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return QMM_ERR_INVALID_ARG;
    if (c->num_pages < 0 || c->num_pages > 0x7FFFFFFF) return QMM_ERR_INVALID_ARG;
    const int64_t strides[6] = {c->k_page_stride, c->k_head_stride, c->k_slot_stride,
                                c->v_page_stride, c->v_head_stride, c->v_slot_stride};
    for (int64_t s : strides)
        if (s < 0 || s % 8 != 0 || s > (1LL << 40)) return QMM_ERR_INVALID_ARG;
    return QMM_OK;
}

// Rows of `elems` elements of `size` bytes, `stride` elements apart.
bool rows_ok(const void* p, int64_t stride, int64_t elems, int size, int64_t n) {
    if (p == nullptr || !aligned(p, 16)) return false;
    return n <= 1 || (stride >= elems && stride <= (1LL << 40) && (stride * size) % 16 == 0);
}

// Arguments of a call, for a descriptor that is valid.
int check_append(const qmm_kv_desc* d, const qmm_kv_cache* cache, const qmm_append_args* a) {
    if (a == nullptr) return QMM_ERR_INVALID_ARG;
    const int chk = check_cache(cache);
    if (chk != QMM_OK) return chk;
    if (a->in_dtype != QMM_IN_F32 && a->in_dtype != QMM_IN_BF16) return QMM_ERR_INVALID_ARG;
    if (a->seqs < 0 || a->seqs > d->max_seqs || a->rows < 0) return QMM_ERR_INVALID_ARG;
    const int64_t tokens = static_cast<int64_t>(a->seqs) * a->rows;
    // the grid has one warp for every few heads of a token
    if (tokens * (d->q_heads + 2 * d->kv_heads) > (1LL << 31)) return QMM_ERR_UNSUPPORTED;
    if (tokens == 0) return QMM_OK;
    const int size = a->in_dtype == QMM_IN_F32 ? 4 : 2;
    const int64_t dq = static_cast<int64_t>(d->q_heads) * d->head_dim, dk = static_cast<int64_t>(d->kv_heads) * d->head_dim;
    if (!rows_ok(a->q, a->q_stride, dq, size, tokens) || !rows_ok(a->k, a->k_stride, dk, size, tokens) ||
        !rows_ok(a->v, a->v_stride, dk, size, tokens) || !rows_ok(a->q_out, a->q_out_stride, dq, 2, tokens))
        return QMM_ERR_INVALID_ARG;
    if (!aligned(a->q_weight, 16) || !aligned(a->k_weight, 16)) return QMM_ERR_INVALID_ARG;
    if (d->rot_dim > 0 && (a->rope == nullptr || !aligned(a->rope, 16) || a->rope_len < 1)) return QMM_ERR_INVALID_ARG;
    if (a->lengths == nullptr || !aligned(a->lengths, 4) || a->page_table == nullptr || !aligned(a->page_table, 4) ||
        !aligned(a->positions, 4))
        return QMM_ERR_INVALID_ARG;
    return QMM_OK;
}

int check_attention(const qmm_kv_desc* d, const qmm_kv_cache* cache, const qmm_attention_args* a) {
    if (a == nullptr) return QMM_ERR_INVALID_ARG;
    const int chk = check_cache(cache);
    if (chk != QMM_OK) return chk;
    const int seqs = a->seqs, rows = a->rows;
    if (seqs < 0 || seqs > d->max_seqs || rows < 0 || rows > d->max_rows) return QMM_ERR_INVALID_ARG;
    const int64_t tokens = static_cast<int64_t>(seqs) * rows;
    if (tokens == 0) return QMM_OK;
    const int64_t row_tiles = (static_cast<int64_t>(rows) * (d->q_heads / d->kv_heads) + 15) / 16;
    if (static_cast<int64_t>(seqs) * d->kv_heads * row_tiles >= (1LL << 30)) return QMM_ERR_UNSUPPORTED;
    const int64_t dq = static_cast<int64_t>(d->q_heads) * d->head_dim;
    if (!rows_ok(a->q, a->q_stride, dq, 2, tokens) || !rows_ok(a->out, a->out_stride, dq, 2, tokens)) return QMM_ERR_INVALID_ARG;
    if (a->page_table == nullptr || !aligned(a->page_table, 4) || a->lengths == nullptr || !aligned(a->lengths, 4))
        return QMM_ERR_INVALID_ARG;
    return QMM_OK;
}

// Makes a plan's device the current one, and at the end of the call the one that was.
class OnDevice {
public:
    explicit OnDevice(int device) {
        int now = 0;
        ok = cudaGetDevice(&now) == cudaSuccess;
        if (ok && now != device) {
            ok = cudaSetDevice(device) == cudaSuccess;
            before_ = now;
        }
    }
    ~OnDevice() {
        if (before_ >= 0) cudaSetDevice(before_);
    }
    OnDevice(const OnDevice&) = delete;
    OnDevice& operator=(const OnDevice&) = delete;
    bool ok;

private:
    int before_ = -1;
};

KvSide side(void* base, int64_t page, int64_t head, int64_t slot) {
    return KvSide{static_cast<uint16_t*>(base), page, head, slot};
}

}  // namespace

extern "C" {

int qmm_kv_validate_desc(const qmm_kv_desc* d) {
    if (d == nullptr) return QMM_ERR_INVALID_ARG;
    if (d->q_heads < 1 || d->kv_heads < 1 || d->head_dim < 1 || d->page_size < 1) return QMM_ERR_INVALID_ARG;
    if (d->q_heads > 65536 || d->q_heads % d->kv_heads != 0) return QMM_ERR_INVALID_ARG;
    if (d->max_seqs < 1 || d->max_seqs > QMM_KV_MAX_SEQS || d->max_pages < 1) return QMM_ERR_INVALID_ARG;
    if (d->max_rows < 1 || d->max_rows > QMM_KV_MAX_ROWS) return QMM_ERR_INVALID_ARG;
    if (d->window < 0 || d->sinks < 0 || d->rot_dim < 0 || d->rot_dim > d->head_dim) return QMM_ERR_INVALID_ARG;
    if (d->interleaved != 0 && d->interleaved != 1) return QMM_ERR_INVALID_ARG;
    if (!std::isfinite(d->scale) || !std::isfinite(d->eps) || d->eps < 0.0f) return QMM_ERR_INVALID_ARG;
    if (static_cast<int64_t>(d->max_pages) * d->page_size > 0x7FFFFFFF - 1024) return QMM_ERR_INVALID_ARG;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return QMM_ERR_UNSUPPORTED;
    if (d->q_heads / d->kv_heads > QMM_KV_MAX_GROUP) return QMM_ERR_UNSUPPORTED;
    if (d->page_size > 1024 || (d->page_size & (d->page_size - 1)) != 0) return QMM_ERR_UNSUPPORTED;
    if (d->rot_dim % 16 != 0) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

size_t qmm_kv_workspace_bytes(const qmm_kv_desc* d) {
    if (qmm_kv_validate_desc(d) != QMM_OK) return 0;
    return attn_workspace(d->head_dim, d->max_rows * (d->q_heads / d->kv_heads)).bytes;
}

int qmm_kv_plan(qmm_kv_plan_t** plan, const qmm_kv_desc* d, void* workspace, size_t ws_bytes) {
    if (plan == nullptr) return QMM_ERR_INVALID_ARG;
    *plan = nullptr;
    const int v = qmm_kv_validate_desc(d);
    if (v != QMM_OK) return v;
    const size_t need = qmm_kv_workspace_bytes(d);
    if (workspace != nullptr && (ws_bytes < need || !aligned(workspace, 256))) return QMM_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QMM_ERR_CUDA;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return QMM_ERR_CUDA;
    if (configure_attention() != cudaSuccess) return QMM_ERR_CUDA;

    struct qmm_kv_plan* p = new (std::nothrow) struct qmm_kv_plan();
    if (p == nullptr) return QMM_ERR_ALLOC;
    p->d = *d;
    p->device = dev;
    p->num_sms = sms;
    p->owns_ws = workspace == nullptr;
    void* ws = workspace;
    if (p->owns_ws && cudaMalloc(&ws, need) != cudaSuccess) {
        delete p;
        return QMM_ERR_ALLOC;
    }
    p->ws = static_cast<uint8_t*>(ws);
    // the error word and the join counters start at zero
    if (cudaMemsetAsync(p->ws, 0, kKvErrBytes + kAttnCounterBytes, 0) != cudaSuccess ||
        cudaStreamSynchronize(0) != cudaSuccess) {
        if (p->owns_ws) cudaFree(p->ws);
        delete p;
        return QMM_ERR_CUDA;
    }
    *plan = p;
    return QMM_OK;
}

int qmm_kv_error(const qmm_kv_plan_t* p, uint32_t* flags) {
    if (p == nullptr || flags == nullptr) return QMM_ERR_INVALID_ARG;
    uint32_t v = 0;
    const OnDevice on(p->device);
    if (!on.ok) return QMM_ERR_CUDA;
    // the plan's calls may be in flight on a stream that the legacy one does not wait for, and later ones must find the word
    // cleared
    if (cudaDeviceSynchronize() != cudaSuccess) return QMM_ERR_CUDA;
    if (cudaMemcpy(&v, p->ws, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return QMM_ERR_CUDA;
    if (v != 0 && (cudaMemset(p->ws, 0, sizeof(v)) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess))
        return QMM_ERR_CUDA;
    *flags = v;
    if (v == 0) return QMM_OK;
    return v & QMM_KV_TIMEOUT ? QMM_ERR_TIMEOUT : QMM_ERR_INVALID_ARG;
}

void qmm_kv_destroy(qmm_kv_plan_t* p) {
    if (p == nullptr) return;
    if (p->owns_ws && p->ws != nullptr) cudaFree(p->ws);
    delete p;
}

int qmm_check_qk_norm_rope_args(const qmm_kv_desc* d, const qmm_kv_cache* cache, const qmm_append_args* a) {
    const int v = qmm_kv_validate_desc(d);
    return v != QMM_OK ? v : check_append(d, cache, a);
}

int qmm_qk_norm_rope(const qmm_kv_plan_t* p, const qmm_kv_cache* cache, const qmm_append_args* a, void* stream) {
    if (p == nullptr) return QMM_ERR_INVALID_ARG;
    const int chk = check_append(&p->d, cache, a);
    if (chk != QMM_OK) return chk;
    if (a->seqs == 0 || a->rows == 0) return QMM_OK;
    const OnDevice on(p->device);
    if (!on.ok) return QMM_ERR_CUDA;
    AppendParams ap;
    ap.k = side(cache->k, cache->k_page_stride, cache->k_head_stride, cache->k_slot_stride);
    ap.v = side(cache->v, cache->v_page_stride, cache->v_head_stride, cache->v_slot_stride);
    ap.in[0] = a->q;
    ap.in[1] = a->k;
    ap.in[2] = a->v;
    ap.in_stride[0] = a->q_stride;
    ap.in_stride[1] = a->k_stride;
    ap.in_stride[2] = a->v_stride;
    ap.q_out = static_cast<uint16_t*>(a->q_out);
    ap.q_out_stride = a->q_out_stride;
    ap.weight[0] = a->q_weight;
    ap.weight[1] = a->k_weight;
    ap.rope = a->rope;
    ap.rope_len = a->rope_len;
    ap.lengths = a->lengths;
    ap.positions = a->positions;
    ap.page_table = a->page_table;
    ap.err = reinterpret_cast<uint32_t*>(p->ws);
    ap.num_pages = cache->num_pages;
    ap.tokens = a->seqs * a->rows;
    ap.rows = a->rows;
    ap.q_heads = p->d.q_heads;
    ap.kv_heads = p->d.kv_heads;
    ap.max_pages = p->d.max_pages;
    ap.page_shift = log2_of(p->d.page_size);
    ap.rot_dim = p->d.rot_dim;
    ap.interleaved = p->d.interleaved;
    ap.eps = p->d.eps;
    return launch_append(p->d.head_dim, a->in_dtype == QMM_IN_F32, ap, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? QMM_OK : QMM_ERR_CUDA;
}

int qmm_check_attention_args(const qmm_kv_desc* d, const qmm_kv_cache* cache, const qmm_attention_args* a) {
    const int v = qmm_kv_validate_desc(d);
    return v != QMM_OK ? v : check_attention(d, cache, a);
}

int qmm_attention(const qmm_kv_plan_t* p, const qmm_kv_cache* cache, const qmm_attention_args* a, void* stream) {
    if (p == nullptr) return QMM_ERR_INVALID_ARG;
    const int chk = check_attention(&p->d, cache, a);
    if (chk != QMM_OK) return chk;
    if (a->seqs == 0 || a->rows == 0) return QMM_OK;
    const OnDevice on(p->device);
    if (!on.ok) return QMM_ERR_CUDA;
    const qmm_kv_desc& d = p->d;
    const int group = d.q_heads / d.kv_heads;
    const AttnWorkspace w = attn_workspace(d.head_dim, d.max_rows * group);
    AttnParams ap;
    ap.k = side(cache->k, cache->k_page_stride, cache->k_head_stride, cache->k_slot_stride);
    ap.v = side(cache->v, cache->v_page_stride, cache->v_head_stride, cache->v_slot_stride);
    ap.q = static_cast<const uint16_t*>(a->q);
    ap.out = static_cast<uint16_t*>(a->out);
    ap.page_table = a->page_table;
    ap.lengths = a->lengths;
    ap.err = reinterpret_cast<uint32_t*>(p->ws);
    ap.counters = reinterpret_cast<uint32_t*>(p->ws + w.counters);
    ap.joins = reinterpret_cast<int4*>(p->ws + w.joins);
    ap.part = reinterpret_cast<float*>(p->ws + w.part);
    ap.part_ml = reinterpret_cast<float*>(p->ws + w.part_ml);
    ap.q_stride = a->q_stride;
    ap.out_stride = a->out_stride;
    ap.num_pages = cache->num_pages;
    ap.seqs = a->seqs;
    ap.rows = a->rows;
    ap.group = group;
    ap.kv_heads = d.kv_heads;
    ap.group_inverse = ((1 << 20) + group - 1) / group;
    ap.row_groups = ap.min_unit = 0;   // set by the launcher for the rows that one CTA holds
    ap.max_pages = d.max_pages;
    ap.page_shift = log2_of(d.page_size);
    ap.window = d.window == 0x7FFFFFFF ? 0 : d.window;   // a window that no position leaves is none
    ap.positions = d.max_pages * d.page_size;
    ap.sinks = d.sinks < ap.positions ? d.sinks : ap.positions;
    ap.query_sign = d.scale < 0.0f ? 0x80008000u : 0u;
    // a scale of 0 would make masked scores of -infinity NaN; one that moves no score does not
    ap.scale_log2 = std::fmax(std::fabs(d.scale), 1e-30f) * 1.4426950408889634f;
    pthread_mutex_lock(&p->launches);
    const cudaError_t e = launch_attention(d.head_dim, ap, p->num_sms, static_cast<cudaStream_t>(stream));
    pthread_mutex_unlock(&p->launches);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

}  // extern "C"
