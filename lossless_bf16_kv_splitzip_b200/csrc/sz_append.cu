// sz_append.cu -- writing a layer's new keys and values into the paged cache:
// head norm, position rotation, page placement and exponent counts in one
// pass over q, k and v.
//
// Mathematics.  For a head x of D channels: y = x * w / sqrt(mean(x^2) + eps);
// the first R channels are R/2 pairs (a, b) turned by pos * f_t:
// (a cos - b sin, b cos + a sin) * scale.  A pair's partner sits R/2 channels
// away (or next to it when interleaved), so a head held 8 channels per lane
// needs one exchange of 16 bytes per lane.
//
// Bound: memory.  Every value is read once and written once, 4 bytes each.
//
// One block per new token: its angles are computed once (a double product,
// reduced by whole turns in double so that a position of millions keeps its
// angle, then a 32-bit sine and cosine) and serve all of its heads.
#include "sz_paged.cuh"

namespace sz {

constexpr int kAppendThreads = 256;
constexpr uint32_t kMaxHeadDim = 256;

// 8 channels of one lane's chunk, partners exchanged: returns y turned.
// `chunk` = channels 8*chunk ..; half layout: the partner chunk lies
// half_chunks away inside the rotated part.
__device__ __forceinline__ void rotate8(float (&y)[8], const float (&partner)[8], const float2 *cs, uint32_t chunk,
                                        uint32_t half_chunks, bool interleaved, float scale) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 c = cs[chunk * 4 + i];
            const float a = y[2 * i], b = y[2 * i + 1];
            y[2 * i] = (a * c.x - b * c.y) * scale;
            y[2 * i + 1] = (b * c.x + a * c.y) * scale;
        }
    } else {
        const bool second = chunk >= half_chunks;
        const uint32_t t0 = (second ? chunk - half_chunks : chunk) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 c = cs[t0 + i];
            const float s = second ? c.y : -c.y;
            y[i] = (y[i] * c.x + partner[i] * s) * scale;
        }
    }
}

template <typename T, int kLanes>  // kLanes lanes hold one head, 8 channels each
__global__ void __launch_bounds__(kAppendThreads) append_kernel(sz_paged_kv kv, sz_append_args a, int32_t *status) {
    __shared__ float2 cs[kMaxHeadDim / 2];
    const uint32_t tid = threadIdx.x;
    const uint32_t D = kv.head_dim;
    const uint32_t chunks = D / 8;

    // ---- the requests' statuses: warps of the grid take one request each
    {
        const uint32_t warps = gridDim.x * (kAppendThreads / 32);
        for (uint32_t r = blockIdx.x * (kAppendThreads / 32) + (tid >> 5); r < kv.n_reqs; r += warps) {
            const Request q = load_request(kv, r);
            sz_status st = q.status;
            if (st == SZ_OK && q.n > q.kv) st = SZ_ERR_INVALID;
            if (st == SZ_OK && q.n > 0) {
                st = check_pages(kv, r, (uint32_t)(q.kv - q.n) / kv.page_tokens, (uint32_t)(q.kv - 1) / kv.page_tokens + 1);
                if (a.d_hists_or_null) {
                    const uint32_t kr = a.d_hist_rows_or_null ? a.d_hist_rows_or_null[r] : r;
                    const uint32_t vr = a.d_hist_rows_or_null ? a.d_hist_rows_or_null[kv.n_reqs + r] : kv.n_reqs + r;
                    if (kr >= a.n_hists || vr >= a.n_hists) st = SZ_ERR_INVALID;
                }
            }
            if ((tid & 31) == 0) status[r] = st;
        }
    }
    if (blockIdx.x >= kv.n_tokens) return;
    const uint32_t token = blockIdx.x;
    const uint32_t r = request_of(kv, token);
    if (r >= kv.n_reqs) return;
    const Request q = load_request(kv, r);
    if (q.status != SZ_OK || q.n > q.kv) return;
    const uint32_t place = (uint32_t)(q.kv - q.n) + (token - (uint32_t)q.q0);
    const int32_t page = page_of(kv, r, place / kv.page_tokens);
    if (page < 0) return;
    uint32_t hk = 0xFFFFFFFFu, hv = 0xFFFFFFFFu;
    if (a.d_hists_or_null) {
        hk = a.d_hist_rows_or_null ? a.d_hist_rows_or_null[r] : r;
        hv = a.d_hist_rows_or_null ? a.d_hist_rows_or_null[kv.n_reqs + r] : kv.n_reqs + r;
        if (hk >= a.n_hists || hv >= a.n_hists) return;
    }
    if (a.rot_dim) {
        const double pos = a.d_positions_or_null ? (double)a.d_positions_or_null[token] : (double)place;
        for (uint32_t t = tid; t < a.rot_dim / 2; t += kAppendThreads) {
            double turns = pos * a.d_freqs_or_null[t] * 0.15915494309189533577;
            turns -= rint(turns);
            float s, c;
            sincospif(2.0f * (float)turns, &s, &c);
            cs[t] = make_float2(c, s);
        }
    }
    __syncthreads();

    const uint32_t lane = tid % kLanes, group = tid / kLanes;
    const uint32_t n_heads = a.q_heads + 2 * kv.heads;
    const uint32_t slot = place % kv.page_tokens;
    const uint32_t half_chunks = a.rot_dim / 16;
    for (uint32_t h0 = 0; h0 < n_heads; h0 += kAppendThreads / kLanes) {
        const uint32_t h = h0 + group;
        const bool live = h < n_heads && lane < chunks;
        const uint16_t *src = nullptr;
        uint16_t *dst = nullptr;
        const uint16_t *w = nullptr;
        bool turn = false, is_k = false, is_v = false;
        if (h < a.q_heads) {
            src = (const uint16_t *)a.d_q_or_null + token * a.q_stride[0] + h * a.q_stride[1];
            dst = (uint16_t *)a.d_q_out + token * a.q_out_stride[0] + h * a.q_out_stride[1];
            w = (const uint16_t *)a.d_q_norm_or_null;
            turn = true;
        } else if (h < a.q_heads + kv.heads) {
            const uint32_t g = h - a.q_heads;
            src = (const uint16_t *)a.d_k + token * a.k_stride[0] + g * a.k_stride[1];
            dst = (uint16_t *)kv.d_k + (uint64_t)page * kv.k_stride[0] + g * kv.k_stride[1] + slot * kv.k_stride[2];
            w = (const uint16_t *)a.d_k_norm_or_null;
            turn = is_k = true;
        } else if (h < n_heads) {
            const uint32_t g = h - a.q_heads - kv.heads;
            src = (const uint16_t *)a.d_v + token * a.v_stride[0] + g * a.v_stride[1];
            dst = (uint16_t *)kv.d_v + (uint64_t)page * kv.v_stride[0] + g * kv.v_stride[1] + slot * kv.v_stride[2];
            is_v = true;
        }
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live) raw = ld_stream_v4(src + lane * 8);
        uint4 out = raw;
        // The exchange needs every lane of the warp: it is made whatever the
        // head, and used by the lanes whose head turns.
        float y[8];
        widen8<T>(raw, y);
        float f = 1.0f;
        {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += y[i] * y[i];
#pragma unroll
            for (int d = kLanes / 2; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            if (w) f = rsqrtf(sum / (float)D + a.eps);
        }
        if (w && live) {
            float ww[8];
            widen8<T>(__ldg((const uint4 *)(w + lane * 8)), ww);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= f * ww[i];
        }
        float partner[8];
        const uint32_t other = lane < half_chunks ? lane + half_chunks : lane - half_chunks;
        if (!a.interleaved && a.rot_dim) {
#pragma unroll
            for (int i = 0; i < 8; ++i) partner[i] = __shfl_sync(0xFFFFFFFFu, y[i], other, kLanes);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) partner[i] = 0.0f;
        }
        if (live && turn) {
            if (lane * 8 < a.rot_dim) rotate8(y, partner, cs, lane, half_chunks, a.interleaved != 0, a.rot_scale);
            if (w || a.rot_dim) out = narrow8<T>(y);
        }
        if (live) {
            *reinterpret_cast<uint4 *>(dst + lane * 8) = out;
            if (a.d_hists_or_null && (is_k || is_v)) {
                uint32_t *row = a.d_hists_or_null + (uint64_t)(is_k ? hk : hv) * 256;
                const uint32_t ws[4] = {out.x, out.y, out.z, out.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    atomicAdd(row + ((ws[i] >> 7) & 0xFFu), 1u);
                    atomicAdd(row + ((ws[i] >> 23) & 0xFFu), 1u);
                }
            }
        }
    }
}

template <typename T>
static cudaError_t launch_append_t(const sz_paged_kv &kv, const sz_append_args &a, int32_t *status, cudaStream_t s) {
    const uint32_t grid = (uint32_t)umax64(kv.n_tokens, div_up(kv.n_reqs, kAppendThreads / 32));
    if (kv.head_dim <= 64)
        append_kernel<T, 8><<<grid, kAppendThreads, 0, s>>>(kv, a, status);
    else if (kv.head_dim <= 128)
        append_kernel<T, 16><<<grid, kAppendThreads, 0, s>>>(kv, a, status);
    else
        append_kernel<T, 32><<<grid, kAppendThreads, 0, s>>>(kv, a, status);
    return cudaGetLastError();
}

cudaError_t launch_append(const sz_paged_kv &kv, const sz_append_args &a, int32_t *status, cudaStream_t s) {
    return kv.dtype == SZ_BF16 ? launch_append_t<__nv_bfloat16>(kv, a, status, s)
                               : launch_append_t<__half>(kv, a, status, s);
}

}  // namespace sz
