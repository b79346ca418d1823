// sz_paged.cuh -- what the operators over the paged cache share: the view of
// the cache and its requests, the checks of a request's arrays, and 16-bit
// conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sz_internal.cuh"

namespace sz {

template <typename T>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ float2 widen(uint32_t w) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
    }
    static __device__ __forceinline__ uint32_t narrow(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <>
struct Half2<__half> {
    using type = __half2;
    static __device__ __forceinline__ float2 widen(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t narrow(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

template <typename T>
__device__ __forceinline__ void widen8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Half2<T>::widen(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
    uint4 v;
    v.x = Half2<T>::narrow(x[0], x[1]);
    v.y = Half2<T>::narrow(x[2], x[3]);
    v.z = Half2<T>::narrow(x[4], x[5]);
    v.w = Half2<T>::narrow(x[6], x[7]);
    return v;
}

// A request's rows and lengths as the device arrays give them.  `status` is
// SZ_OK or why the request is refused; a refused request has no rows.
struct Request {
    int32_t q0;    // first row
    int32_t n;     // rows
    int32_t kv;    // cached tokens, the new ones included
    sz_status status;
};
__device__ __forceinline__ Request load_request(const sz_paged_kv &kv, uint32_t r) {
    Request q;
    const int32_t a = __ldg(kv.d_q_begin + r), b = __ldg(kv.d_q_begin + r + 1);
    q.q0 = a;
    q.n = b - a;
    q.kv = __ldg(kv.d_kv_len + r);
    q.status = SZ_OK;
    if (a < 0 || b < a || (uint64_t)b > kv.n_tokens || q.kv < 0)
        q.status = SZ_ERR_INVALID;
    else if ((uint64_t)q.kv > (uint64_t)kv.max_pages * kv.page_tokens)
        q.status = SZ_ERR_CAPACITY;
    if (q.status != SZ_OK) q.n = q.kv = 0;
    return q;
}

// The request that owns row `token`, or n_reqs: the largest r with
// q_begin[r] <= token, if the row lies in it.
__device__ __forceinline__ uint32_t request_of(const sz_paged_kv &kv, uint32_t token) {
    uint32_t lo = 0, hi = kv.n_reqs;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (__ldg(kv.d_q_begin + mid) <= (int32_t)token) lo = mid; else hi = mid;
    }
    if (kv.n_reqs == 0 || __ldg(kv.d_q_begin + lo) > (int32_t)token || __ldg(kv.d_q_begin + lo + 1) <= (int32_t)token)
        return kv.n_reqs;
    return lo;
}

// Page of token position `pos` of request r, or -1 when its number lies
// outside the pool (pos must be inside the request's table row).
__device__ __forceinline__ int32_t page_of(const sz_paged_kv &kv, uint32_t r, uint32_t index) {
    const int32_t p = __ldg(kv.d_page_table + (uint64_t)r * kv.table_stride + index);
    return (p < 0 || (uint64_t)p >= kv.n_pages) ? -1 : p;
}

// Status of request r over its pages [first, end), by one warp: lanes look
// at different pages and agree.
__device__ __forceinline__ sz_status check_pages(const sz_paged_kv &kv, uint32_t r, uint32_t first, uint32_t end) {
    bool bad = false;
    for (uint32_t i = first + (threadIdx.x & 31); i < end; i += 32) bad |= page_of(kv, r, i) < 0;
    return __any_sync(0xFFFFFFFFu, bad) ? SZ_ERR_INVALID : SZ_OK;
}

// Host checks shared by the two entry points: null pointers, sizes,
// alignment, and strides that keep values apart.
sz_status check_paged_kv(const sz_paged_kv *kv);
// Rows of n heads of kv->head_dim values: a pointer and strides that vector
// accesses allow.
sz_status check_rows(const sz_paged_kv *kv, const void *p, const uint64_t (&stride)[2], uint32_t heads);

}  // namespace sz
