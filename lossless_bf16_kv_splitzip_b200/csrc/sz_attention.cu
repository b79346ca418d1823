// sz_attention.cu -- softmax attention of new tokens over the paged cache.
//
// Mathematics.  A row's softmax is carried over the keys in one pass with a
// running maximum m, sum l and accumulator o: a key with score s changes them
// to m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') +
// e^(s - m') v; two such triples over different keys join the same way.
// Exponentials are taken base 2 of scores scaled by log2(e).
#include "sz_paged.cuh"

namespace sz {

constexpr int kGeneralThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------ any shape
// One block per (new token, query head), any page size and head size: groups
// of kLanes lanes (8 channels each) take keys in turn, each with its own
// running softmax, joined at the end.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kGeneralThreads) attention_any_kernel(sz_paged_kv kv, sz_attention_args a, int32_t *status) {
    constexpr int kGroups = kGeneralThreads / kLanes;
    __shared__ float part[kGroups][kLanes * 8 + 2];
    const uint32_t tid = threadIdx.x;
    const uint32_t head = blockIdx.y;
    if (head == 0) {  // the requests' statuses: warps of the row of blocks take one request each
        const uint32_t warps = gridDim.x * (kGeneralThreads / 32);
        for (uint32_t r = blockIdx.x * (kGeneralThreads / 32) + (tid >> 5); r < kv.n_reqs; r += warps) {
            const Request q = load_request(kv, r);
            sz_status st = q.status;
            if (st == SZ_OK && q.n > 0 && q.kv > 0) {
                const int32_t first = a.window ? max(0, q.kv - q.n - (int32_t)umin32(a.window, 0x7FFFFFFFu) + 1) : 0;
                st = check_pages(kv, r, (uint32_t)first / kv.page_tokens, (uint32_t)(q.kv - 1) / kv.page_tokens + 1);
            }
            if ((tid & 31) == 0) status[r] = st;
        }
    }
    if (blockIdx.x >= kv.n_tokens) return;
    const uint32_t token = blockIdx.x;
    const uint32_t r = request_of(kv, token);
    if (r >= kv.n_reqs) return;
    const Request q = load_request(kv, r);
    if (q.status != SZ_OK) return;
    const uint32_t lane = tid % kLanes, group = tid / kLanes;
    const uint32_t chunks = kv.head_dim / 8;
    const uint32_t kvh = head / (a.q_heads / kv.heads);
    const int32_t p = q.kv - q.n + (int32_t)(token - (uint32_t)q.q0);
    const int32_t end = a.causal ? min(q.kv, p + 1) : q.kv;
    const int32_t begin = a.window ? max(0, (int32_t)max((int64_t)0, (int64_t)p - a.window + 1)) : 0;
    const bool live = lane < chunks;
    float x[8] = {};
    if (live) widen8<T>(*(const uint4 *)((const uint16_t *)a.d_q + token * a.q_stride[0] + head * a.q_stride[1] + lane * 8), x);
    const float scale = a.scale * kLog2e;
    float m = -INFINITY, l = 0.0f, o[8] = {};
    for (int32_t j0 = begin; j0 < end; j0 += kGroups) {
        const int32_t j = j0 + (int32_t)group;
        int32_t page = -1;
        if (j < end) page = page_of(kv, r, (uint32_t)j / kv.page_tokens);
        const uint32_t slot = (uint32_t)j % kv.page_tokens;
        float k[8] = {}, v[8] = {};
        if (live && page >= 0) {
            widen8<T>(*(const uint4 *)((const uint16_t *)kv.d_k + (uint64_t)page * kv.k_stride[0] + kvh * kv.k_stride[1] +
                                       slot * kv.k_stride[2] + lane * 8), k);
            widen8<T>(*(const uint4 *)((const uint16_t *)kv.d_v + (uint64_t)page * kv.v_stride[0] + kvh * kv.v_stride[1] +
                                       slot * kv.v_stride[2] + lane * 8), v);
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[i] * k[i];
#pragma unroll
        for (int d = kLanes / 2; d >= 1; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        if (j < end && page >= 0) {
            s *= scale;
            const float m1 = fmaxf(m, s);
            const float keep = m1 == m ? 1.0f : exp2f(m - m1);  // also the first key, and a score of -inf
            const float e = s == -INFINITY ? 0.0f : exp2f(s - m1);
            l = l * keep + e;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = o[i] * keep + e * v[i];
            m = m1;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[group][lane * 8 + i] = o[i];
    if (lane == 0) {
        part[group][kLanes * 8] = m;
        part[group][kLanes * 8 + 1] = l;
    }
    __syncthreads();
    if (group != 0) return;
    const bool any = begin < end;
    float mm = -INFINITY;
    for (int g = 0; g < kGroups; ++g) mm = fmaxf(mm, part[g][kLanes * 8]);
    float ll = 0.0f, oo[8] = {};
    for (int g = 0; g < kGroups; ++g) {
        const float lg = part[g][kLanes * 8 + 1];
        if (lg == 0.0f) continue;  // a group without keys
        const float f = exp2f(part[g][kLanes * 8] - mm);
        ll += lg * f;
#pragma unroll
        for (int i = 0; i < 8; ++i) oo[i] += part[g][lane * 8 + i] * f;
    }
    const float inv = any ? 1.0f / ll : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) oo[i] = any ? oo[i] * inv : 0.0f;
    if (live)
        *(uint4 *)((uint16_t *)a.d_out + token * a.out_stride[0] + head * a.out_stride[1] + lane * 8) = narrow8<T>(oo);
    if (a.d_lse_or_null && lane == 0)
        a.d_lse_or_null[(uint64_t)token * a.q_heads + head] = any ? (mm + log2f(ll)) * kLn2 : -INFINITY;
}

template <typename T>
static cudaError_t launch_any_t(const sz_paged_kv &kv, const sz_attention_args &a, int32_t *status, cudaStream_t s) {
    const dim3 grid((uint32_t)umax64(kv.n_tokens, div_up(kv.n_reqs, kGeneralThreads / 32)), a.q_heads);
    if (kv.head_dim <= 64)
        attention_any_kernel<T, 8><<<grid, kGeneralThreads, 0, s>>>(kv, a, status);
    else if (kv.head_dim <= 128)
        attention_any_kernel<T, 16><<<grid, kGeneralThreads, 0, s>>>(kv, a, status);
    else
        attention_any_kernel<T, 32><<<grid, kGeneralThreads, 0, s>>>(kv, a, status);
    return cudaGetLastError();
}

cudaError_t launch_attention(const sz_paged_kv &kv, const sz_attention_args &a, int32_t *status, cudaStream_t s) {
    return kv.dtype == SZ_BF16 ? launch_any_t<__nv_bfloat16>(kv, a, status, s) : launch_any_t<__half>(kv, a, status, s);
}

}  // namespace sz
