// sz_paged_api.cu -- the C entry points of the operators over the paged cache:
// argument checks and launches.  Host code only; it allocates nothing and
// never synchronises the caller's stream.
#include "sz_paged.cuh"

namespace sz {

cudaError_t launch_append(const sz_paged_kv &kv, const sz_append_args &a, int32_t *status, int sms, cudaStream_t s);
cudaError_t launch_attention(const sz_paged_kv &kv, const sz_attention_args &a, int32_t *status, void *ws, const DeviceInfo &dev,
                             cudaStream_t s);
uint64_t attention_workspace(uint32_t head_dim);

namespace {

constexpr uint64_t kMaxRows = 1ull << 30;       // rows, requests and positions: sums of two fit in an int32
constexpr uint64_t kMaxPages = 0x7FFFFFFFull;   // page numbers are int32
constexpr uint64_t kMaxStride = 1ull << 39;     // elements: a tensor map's strides stay below 2^40 bytes
constexpr uint32_t kMaxHeads = 65535;           // a grid dimension

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Strides of a pool of n[0] pages x n[1] heads x n[2] tokens of `dim` values:
// multiples of 8 that keep every value apart, the dimensions nesting inside
// one another in some order.
sz_status check_pool(const uint64_t (&stride)[3], const uint64_t (&n)[3], uint64_t dim) {
    bool used[3] = {};
    uint64_t extent = dim;  // elements the dimensions taken so far span
    for (int step = 0; step < 3; ++step) {
        int best = -1;
        for (int i = 0; i < 3; ++i)
            if (!used[i] && n[i] > 1 && (best < 0 || stride[i] < stride[best])) best = i;
        if (best < 0) break;
        used[best] = true;
        if (stride[best] & 7) return SZ_ERR_ALIGN;
        if (stride[best] < extent) return SZ_ERR_INVALID;
        if (stride[best] >= kMaxStride) return SZ_ERR_TOO_LARGE;
        extent += stride[best] * (n[best] - 1);
        if (extent >= 1ull << 62) return SZ_ERR_TOO_LARGE;
    }
    return SZ_OK;
}

}  // namespace

sz_status check_rows(const sz_paged_kv *kv, const void *p, const uint64_t (&stride)[2], uint32_t heads) {
    if (kv->n_tokens == 0) return SZ_OK;
    if (!p) return SZ_ERR_NULL;
    if (!aligned(p, 16)) return SZ_ERR_ALIGN;
    if ((kv->n_tokens > 1 && (stride[0] & 7)) || (heads > 1 && (stride[1] & 7))) return SZ_ERR_ALIGN;
    if ((kv->n_tokens > 1 && stride[0] >= kMaxStride) || (heads > 1 && stride[1] >= kMaxStride)) return SZ_ERR_TOO_LARGE;
    return SZ_OK;
}

// Rows that are written: tokens and heads may lie in either order, but apart.
static sz_status check_out_rows(const sz_paged_kv *kv, const void *p, const uint64_t (&stride)[2], uint32_t heads) {
    if (const sz_status st = check_rows(kv, p, stride, heads)) return st;
    const uint64_t s3[3] = {stride[0], stride[1], 0}, n3[3] = {kv->n_tokens, heads, 1};
    return check_pool(s3, n3, kv->head_dim);
}

sz_status check_paged_kv(const sz_paged_kv *kv) {
    if (!kv) return SZ_ERR_NULL;
    if (kv->n_reqs > kMaxRows || kv->n_tokens > kMaxRows || kv->n_pages > kMaxPages) return SZ_ERR_TOO_LARGE;
    if (kv->page_tokens > kMaxRows || (uint64_t)kv->max_pages * kv->page_tokens > kMaxRows) return SZ_ERR_TOO_LARGE;
    if (kv->dtype != SZ_BF16 && kv->dtype != SZ_FP16) return SZ_ERR_INVALID;
    if (kv->heads == 0 || kv->heads > kMaxHeads || kv->page_tokens == 0) return SZ_ERR_INVALID;
    if (kv->head_dim == 0 || kv->head_dim > 256 || kv->head_dim % 8) return SZ_ERR_INVALID;
    if (kv->n_reqs > 0) {
        if (!kv->d_q_begin || !kv->d_kv_len) return SZ_ERR_NULL;
        if (kv->max_pages > 0 && !kv->d_page_table) return SZ_ERR_NULL;
        if (!aligned(kv->d_q_begin, 4) || !aligned(kv->d_kv_len, 4) || !aligned(kv->d_page_table, 4)) return SZ_ERR_ALIGN;
        if (kv->n_reqs > 1 && kv->table_stride < kv->max_pages) return SZ_ERR_INVALID;
    }
    if (kv->n_pages > 0 && (!kv->d_k || !kv->d_v)) return SZ_ERR_NULL;
    if (!aligned(kv->d_k, 16) || !aligned(kv->d_v, 16)) return SZ_ERR_ALIGN;
    const uint64_t n[3] = {kv->n_pages, kv->heads, kv->page_tokens};
    if (const sz_status st = check_pool(kv->k_stride, n, kv->head_dim)) return st;
    return check_pool(kv->v_stride, n, kv->head_dim);
}

}  // namespace sz

using namespace sz;

extern "C" {

sz_status sz_append_kv(const sz_paged_kv *kv, const sz_append_args *a, int32_t *d_status, void *stream) {
    if (!a) return SZ_ERR_NULL;
    if (const sz_status st = check_paged_kv(kv)) return st;
    if (kv->n_reqs == 0) return SZ_OK;
    if (!d_status) return SZ_ERR_NULL;
    if (const sz_status st = check_rows(kv, a->d_k, a->k_stride, kv->heads)) return st;
    if (const sz_status st = check_rows(kv, a->d_v, a->v_stride, kv->heads)) return st;
    if (a->q_heads > kMaxHeads) return SZ_ERR_INVALID;
    if (a->q_heads > 0) {
        if (const sz_status st = check_rows(kv, a->d_q_or_null, a->q_stride, a->q_heads)) return st;
        if (const sz_status st = check_out_rows(kv, a->d_q_out, a->q_out_stride, a->q_heads)) return st;
    }
    if (a->rot_dim % 16 || a->rot_dim > kv->head_dim) return SZ_ERR_INVALID;
    if (a->rot_dim > 0 && !a->d_freqs_or_null) return SZ_ERR_NULL;
    if (a->n_hists > 0 && !a->d_hists_or_null) return SZ_ERR_NULL;
    if (!aligned(a->d_q_norm_or_null, 16) || !aligned(a->d_k_norm_or_null, 16) || !aligned(a->d_freqs_or_null, 8) ||
        !aligned(a->d_positions_or_null, 8) || !aligned(a->d_hists_or_null, 4) || !aligned(a->d_hist_rows_or_null, 4) ||
        !aligned(d_status, 4))
        return SZ_ERR_ALIGN;
    DeviceInfo dev;
    if (const sz_status st = device_info(dev)) return st;
    const cudaError_t e = launch_append(*kv, *a, d_status, dev.sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SZ_OK : SZ_ERR_CUDA;
}

sz_status sz_plan_attention(uint32_t head_dim, uint64_t *workspace_bytes) {
    if (!workspace_bytes) return SZ_ERR_NULL;
    if (head_dim == 0 || head_dim > 256 || head_dim % 8) return SZ_ERR_INVALID;
    *workspace_bytes = attention_workspace(head_dim);
    return SZ_OK;
}

sz_status sz_paged_attention(const sz_paged_kv *kv, const sz_attention_args *a, int32_t *d_status, void *d_ws,
                             uint64_t ws_bytes, void *stream) {
    if (!a) return SZ_ERR_NULL;
    if (const sz_status st = check_paged_kv(kv)) return st;
    if (kv->n_reqs == 0) return SZ_OK;
    if (!d_status || !d_ws) return SZ_ERR_NULL;
    if (a->q_heads == 0 || a->q_heads > kMaxHeads || a->q_heads % kv->heads) return SZ_ERR_INVALID;
    if (a->window > 0 && !a->causal) return SZ_ERR_INVALID;
    if (const sz_status st = check_rows(kv, a->d_q, a->q_stride, a->q_heads)) return st;
    if (const sz_status st = check_out_rows(kv, a->d_out, a->out_stride, a->q_heads)) return st;
    if (!aligned(a->d_lse_or_null, 4) || !aligned(d_ws, 16) || !aligned(d_status, 4)) return SZ_ERR_ALIGN;
    uint64_t need = 0;
    if (const sz_status st = sz_plan_attention(kv->head_dim, &need)) return st;
    if (ws_bytes < need) return SZ_ERR_WORKSPACE;
    DeviceInfo dev;
    if (const sz_status st = device_info(dev)) return st;
    const cudaError_t e = launch_attention(*kv, *a, d_status, d_ws, dev, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SZ_OK : SZ_ERR_CUDA;
}

}  // extern "C"
