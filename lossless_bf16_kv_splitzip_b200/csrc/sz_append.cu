// sz_append.cu -- writing a layer's new keys and values into the paged cache:
// head norm, position rotation, page placement and exponent counts in one
// pass over q, k and v.
//
// Mathematics.  For a head x of D channels: y = x * w / sqrt(mean(x^2) + eps);
// the first R channels are R/2 pairs (a, b) turned by pos * f_t:
// (a cos - b sin, b cos + a sin) * scale.  A lane holds two runs of four
// channels that are four whole pairs -- R/2 channels apart, or side by side
// when pairs are adjacent -- so that turning needs no exchange between lanes.
//
// Bound: memory.  Every value is read once and written once, 4 bytes each:
// 4,096 tokens of 32 + 8 + 8 heads of 128 with norms take 22.6 us, 4.4 TB/s
// (68 % of a copy; 4 us of them a launch of little work takes as well), 4,096
// of 64 + 8 + 8 heads 33.7 us, 5.0 TB/s (76 %), one token for each of 64
// requests 4.6 us, which is latency.  With counts, 2,052 tokens on average of
// 3 requests, 8 + 8 heads, take 17.7 us, 2.8 TB/s: not the atomics, which the
// histogram kernel issues at 4 us for as many values, but a warp that counts one
// token before it loads its next, four such rounds in a row, and the clearing
// and folding of 32 KB around them.
// A warp takes one token and a run of its heads (D = 128: two heads at a
// time, two 8-byte loads per lane), kBatch heads' loads under way per lane;
// nothing but the counts needs other warps.  The first loads are issued before
// the token's request, page and angles are looked up, which is a chain of
// dependent loads.
// A token's angles are computed once per warp (a double product, reduced by
// whole turns in double so that a position of millions keeps its angle, then
// a 32-bit sine and cosine) and serve all of its heads.
#include <type_traits>

#include "sz_paged.cuh"

namespace sz {

// Warps per block: few without counts, so that blocks spread evenly over the
// SMs; with counts as many threads as bins.
constexpr int kAppendWarps = 4, kCountWarps = 8;
constexpr uint32_t kMaxHeadDim = 256;
// Blocks per SM that the registers allow: without counts 72 registers and
// nearly no spills for 7 (6 or 8 blocks took 4 to 25 % longer on chunks), with
// counts 3 with their 32 KB of columns each.
constexpr int kAppendBlocks = 7, kCountBlocks = 3;

struct AppendArgs {
    sz_paged_kv kv;
    sz_append_args a;
    int32_t *status;
    uint32_t tokens_per_block;
    uint32_t slice_heads;  // heads a block takes of each of its tokens (without counts)
};

// The request that owns row `token`, or n_reqs, by one warp: 32 entries of
// q_begin are compared at a time, so that n requests take log32(n) rounds.
__device__ __forceinline__ uint32_t warp_request_of(const sz_paged_kv &kv, uint32_t token, uint32_t lane) {
    uint32_t lo = 0, n = kv.n_reqs;  // the answer, if any, is in [lo, lo + n)
    while (n > 1) {
        const uint32_t step = (n + 31) / 32;
        const uint32_t at = lo + lane * step;
        const bool before = lane * step < n && __ldg(kv.d_q_begin + at) <= (int32_t)token;
        const uint32_t hits = __ballot_sync(0xFFFFFFFFu, before);
        if (hits == 0) return kv.n_reqs;
        const uint32_t last = 31 - __clz(hits);  // the largest sample at or before the token
        n = umin32(step, n - last * step);
        lo += last * step;
    }
    return lo;
}

// Where a token's keys and values go.
struct Place {
    uint32_t r;     // n_reqs: nowhere
    uint32_t place;  // position in the cache
    int32_t page;
    uint32_t slot;
};
__device__ __forceinline__ Place place_in(const AppendArgs &p, uint32_t r, const Request &q, uint32_t token) {
    Place x;
    x.r = r;
    x.place = (uint32_t)(q.kv - q.n) + (token - (uint32_t)q.q0);
    x.slot = x.place % p.kv.page_tokens;
    x.page = page_of(p.kv, r, x.place / p.kv.page_tokens);
    if (x.page < 0) x.r = p.kv.n_reqs;
    return x;
}
// Whether row `token` is one of request q's, and q one that can be written.
__device__ __forceinline__ bool owns(const Request &q, uint32_t token) {
    return q.status == SZ_OK && q.n <= q.kv && token >= (uint32_t)q.q0 && token < (uint32_t)(q.q0 + q.n);
}
__device__ __forceinline__ Place token_place(const AppendArgs &p, uint32_t token, uint32_t lane) {
    Place x;
    x.r = warp_request_of(p.kv, token, lane);
    x.page = -1;
    x.place = x.slot = 0;
    if (x.r >= p.kv.n_reqs) return x;
    const Request q = load_request(p.kv, x.r);
    if (owns(q, token)) return place_in(p, x.r, q, token);
    x.r = p.kv.n_reqs;
    return x;
}

// Rows of the histograms that request r's keys and values go to; false when
// one is out of range.
__device__ __forceinline__ bool hist_rows(const AppendArgs &p, uint32_t r, uint32_t &k_row, uint32_t &v_row) {
    k_row = p.a.d_hist_rows_or_null ? p.a.d_hist_rows_or_null[r] : r;
    v_row = p.a.d_hist_rows_or_null ? p.a.d_hist_rows_or_null[p.kv.n_reqs + r] : p.kv.n_reqs + r;
    return k_row < p.a.n_hists && v_row < p.a.n_hists;
}

// Exponent counts of a block: 256 bins x 32 lane columns, bin-major, so that
// the lanes of a warp never meet in a bank whatever exponents they hold.
__device__ __forceinline__ void count2(uint2 v, uint32_t column) {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // the exponent sits in bits 7..14 of each half: exponent * 128 is the row's byte offset
        asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(column + (w[i] & 0x7F80u)) : "memory");
        asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(column + ((w[i] >> 16) & 0x7F80u)) : "memory");
    }
}

template <typename T>
__device__ __forceinline__ void widen4(uint2 v, float (&x)[4]) {
    const float2 a = Half2<T>::widen(v.x), b = Half2<T>::widen(v.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
template <typename T>
__device__ __forceinline__ uint2 narrow4(float a, float b, float c, float d) {
    return make_uint2(Half2<T>::narrow(a, b), Half2<T>::narrow(c, d));
}
__device__ __forceinline__ uint2 ld_stream_v2(const void *p) { return __ldcs(reinterpret_cast<const uint2 *>(p)); }

// One token's heads [h_begin, h_end) by one warp; kLanes lanes hold one head.
// Its request is looked up unless known (known_r < n_reqs).
template <typename T, int kLanes, bool kAdjacent, bool kCount>
__device__ __forceinline__ void append_token(const AppendArgs &p, uint32_t token, uint32_t h_begin, uint32_t h_end, uint32_t lane,
                                             float2 *cs, uint32_t column, uint32_t known_r, const Request &known) {
    constexpr uint32_t kHeads = 32 / kLanes;  // at a time
    // Head groups whose loads a warp has under way: two where many warps run
    // (with four a decode step took 4.7 us instead of 4.3), four next to the
    // counts' 24 warps per SM (17.9 us, with two 19.1).
    constexpr int kBatch = kCount ? 4 : 2;
    const sz_paged_kv &kv = p.kv;
    const sz_append_args &a = p.a;
    const uint32_t D = kv.head_dim, l = lane % kLanes, group = lane / kLanes;
    const uint32_t pairs = a.rot_dim / 2, turning = pairs / 4;  // lanes whose channels turn
    const bool in_head = l * 8 < D, turns_here = l < turning;
    // this lane's two runs of four channels
    const uint32_t c0 = kAdjacent ? l * 8 : turns_here ? l * 4 : l * 8;
    const uint32_t delta = kAdjacent || !turns_here ? 4 : pairs, c1 = c0 + delta;
    float cos4[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sin4[4] = {};
    Place at;
    at.r = kv.n_reqs + 1;  // not looked up
    at.page = at.slot = at.place = 0;
#pragma unroll 1
    for (uint32_t segment = 0; segment < 3; ++segment) {  // queries, keys, values
        const uint32_t s_begin = segment == 0 ? 0 : a.q_heads + (segment - 1) * kv.heads;
        const uint32_t s_heads = segment == 0 ? a.q_heads : kv.heads;
        const uint32_t from = h_begin > s_begin ? h_begin - s_begin : 0;
        const uint32_t to = h_end > s_begin ? umin32(h_end - s_begin, s_heads) : 0;  // of the segment's heads
        if (from >= to) continue;
        const uint16_t *src = (const uint16_t *)(segment == 0 ? a.d_q_or_null : segment == 1 ? a.d_k : a.d_v);
        const uint64_t *const ss = segment == 0 ? a.q_stride : segment == 1 ? a.k_stride : a.v_stride;
        const uint64_t src_step = ss[1] * kHeads;
        src += token * ss[0] + (from + group) * ss[1] + c0;
        const uint16_t *const w = (const uint16_t *)(segment == 0 ? a.d_q_norm_or_null : segment == 1 ? a.d_k_norm_or_null : nullptr);
        const bool turn = pairs && segment < 2;
        uint2 wu_raw = make_uint2(0, 0), wv_raw = wu_raw;
        if (w && in_head) {
            wu_raw = __ldg((const uint2 *)(w + c0));
            wv_raw = __ldg((const uint2 *)(w + c1));
        }
        uint16_t *dst = nullptr;
        uint64_t dst_step = 0;
        // kBatch heads per lane; `checked`: some of them, or some lanes, may
        // lie outside
        auto batch = [&](uint32_t h0, auto checked) {
            constexpr bool kChecked = decltype(checked)::value;
            uint2 x0[kBatch], x1[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (!kChecked || (h0 + i * kHeads + group < to && in_head)) {
                    x0[i] = ld_stream_v2(src);
                    x1[i] = ld_stream_v2(src + delta);
                } else {
                    x0[i] = x1[i] = make_uint2(0, 0);
                }
                src += src_step;
            }
            if (at.r > kv.n_reqs) {  // once, with loads under way
                at = known_r < kv.n_reqs ? place_in(p, known_r, known, token) : token_place(p, token, lane);
                if (at.r < kv.n_reqs && turn) {
                    const double pos = a.d_positions_or_null ? (double)a.d_positions_or_null[token] : (double)at.place;
                    __syncwarp();  // the last token's angles have been read
                    for (uint32_t t = lane; t < pairs; t += 32) {
                        double turns = pos * a.d_freqs_or_null[t] * 0.15915494309189533577;
                        turns -= rint(turns);
                        float sn, cn;
                        sincospif(2.0f * (float)turns, &sn, &cn);
                        cs[t] = make_float2(cn * a.rot_scale, sn * a.rot_scale);
                    }
                    __syncwarp();
                    if (turns_here)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 y = cs[l * 4 + i];
                            cos4[i] = y.x;
                            sin4[i] = y.y;
                        }
                }
            }
            if (at.r >= kv.n_reqs) return;
            if (dst == nullptr) {
                if (segment == 0) {
                    dst = (uint16_t *)a.d_q_out + token * a.q_out_stride[0] + (from + group) * a.q_out_stride[1] + c0;
                    dst_step = a.q_out_stride[1] * kHeads;
                } else {
                    const uint64_t *const ds = segment == 1 ? kv.k_stride : kv.v_stride;
                    dst = (uint16_t *)(segment == 1 ? kv.d_k : kv.d_v) + (uint64_t)at.page * ds[0] + at.slot * ds[2] + (from + group) * ds[1] + c0;
                    dst_step = ds[1] * kHeads;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (kChecked && h0 + i * kHeads >= to) break;
                uint2 y0 = x0[i], y1 = x1[i];
                if (w || turn) {
                    float u[4], v[4];
                    widen4<T>(y0, u);
                    widen4<T>(y1, v);
                    if (w) {
                        float sum = 0.0f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum += u[e] * u[e] + v[e] * v[e];
#pragma unroll
                        for (int d = kLanes / 2; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
                        const float f = rsqrtf(sum / (float)D + a.eps);
                        float wu[4], wv[4];
                        widen4<T>(wu_raw, wu);
                        widen4<T>(wv_raw, wv);
#pragma unroll
                        for (int e = 0; e < 4; ++e) u[e] *= f * wu[e], v[e] *= f * wv[e];
                    }
                    if (turn && turns_here) {
                        // pair i: (u[i], v[i]), or neighbours in u then v
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float &a_ = kAdjacent ? (e < 2 ? u[2 * e] : v[2 * e - 4]) : u[e];
                            float &b_ = kAdjacent ? (e < 2 ? u[2 * e + 1] : v[2 * e - 3]) : v[e];
                            const float turned = a_ * cos4[e] - b_ * sin4[e];
                            b_ = b_ * cos4[e] + a_ * sin4[e];
                            a_ = turned;
                        }
                    }
                    y0 = narrow4<T>(u[0], u[1], u[2], u[3]);
                    y1 = narrow4<T>(v[0], v[1], v[2], v[3]);
                }
                if (!kChecked || (h0 + i * kHeads + group < to && in_head)) {
                    *reinterpret_cast<uint2 *>(dst) = y0;
                    *reinterpret_cast<uint2 *>(dst + delta) = y1;
                    if (kCount && segment > 0) {
                        count2(y0, column);
                        count2(y1, column);
                    }
                }
                dst += dst_step;
            }
        };
        uint32_t h0 = from;
        if (D == kLanes * 8)
            for (; h0 + kBatch * kHeads <= to; h0 += kBatch * kHeads) batch(h0, std::false_type{});
        for (; h0 < to; h0 += kBatch * kHeads) batch(h0, std::true_type{});
        if (at.r >= kv.n_reqs) return;
    }
}

template <typename T, int kLanes, bool kAdjacent, bool kCount>
__global__ void __launch_bounds__(32 * (kCount ? kCountWarps : kAppendWarps), kCount ? kCountBlocks : kAppendBlocks) append_kernel(const __grid_constant__ AppendArgs p) {
    constexpr uint32_t kWarps = kCount ? kCountWarps : kAppendWarps, kThreads = 32 * kWarps;
    __shared__ float2 cs[kWarps][kMaxHeadDim / 2];
    __shared__ uint32_t columns[kCount ? 256 * 32 : 1];
    const sz_paged_kv &kv = p.kv;
    const uint32_t tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

    // ---- the requests' statuses: warps of the first row of blocks take one each
    if (blockIdx.y == 0) {
        for (uint32_t r = blockIdx.x * kWarps + wid; r < kv.n_reqs; r += gridDim.x * kWarps) {
            const Request q = load_request(kv, r);
            sz_status st = q.status;
            uint32_t k_row, v_row;
            if (st == SZ_OK && q.n > q.kv) st = SZ_ERR_INVALID;
            if (st == SZ_OK && q.n > 0) {
                st = check_pages(kv, r, (uint32_t)(q.kv - q.n) / kv.page_tokens, (uint32_t)(q.kv - 1) / kv.page_tokens + 1);
                if (kCount && !hist_rows(p, r, k_row, v_row)) st = SZ_ERR_INVALID;
            }
            if (lane == 0) p.status[r] = st;
        }
    }
    const uint32_t t_begin = blockIdx.x * p.tokens_per_block;
    const uint32_t t_end = (uint32_t)umin64(kv.n_tokens, (uint64_t)t_begin + p.tokens_per_block);
    const uint32_t all = p.a.q_heads + 2 * kv.heads;
    if constexpr (!kCount) {
        const uint32_t h_begin = blockIdx.y * p.slice_heads, h_end = umin32(all, h_begin + p.slice_heads);
        for (uint32_t t = t_begin + wid; t < t_end; t += kWarps)
            append_token<T, kLanes, kAdjacent, false>(p, t, h_begin, h_end, lane, cs[wid], 0, kv.n_reqs, Request{});
    } else {
        // Block rows: keys, values and (if any) queries.  The counts of a
        // request's tokens are added to its row before the next request's.
        const bool is_q = blockIdx.y == 2, is_v = blockIdx.y == 1;
        const uint32_t h_begin = is_q ? 0 : p.a.q_heads + (is_v ? kv.heads : 0);
        const uint32_t h_end = is_q ? p.a.q_heads : h_begin + kv.heads;
        if (!is_q) {
            for (uint32_t i = tid; i < 256 * 32 / 4; i += kThreads) reinterpret_cast<uint4 *>(columns)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
        }
        const uint32_t column = smem_u32(columns) + 4 * lane;
        uint32_t t = t_begin;
        while (t < t_end) {  // the same run of tokens in every warp
            const uint32_t r = warp_request_of(kv, t, lane);
            uint32_t stop = t + 1, k_row = 0, v_row = 0;  // alone, if it is a row of no request
            bool counted = false;
            Request q{};
            if (r < kv.n_reqs) {
                q = load_request(kv, r);
                if (owns(q, t)) {
                    stop = umin32(t_end, (uint32_t)(q.q0 + q.n));
                    counted = hist_rows(p, r, k_row, v_row);
                }
            }
            if (counted) {
                for (uint32_t i = t + wid; i < stop; i += kWarps)
                    if (is_q)
                        append_token<T, kLanes, kAdjacent, false>(p, i, h_begin, h_end, lane, cs[wid], 0, r, q);
                    else
                        append_token<T, kLanes, kAdjacent, true>(p, i, h_begin, h_end, lane, cs[wid], column, r, q);
                if (!is_q) {
                    __syncthreads();
                    uint32_t sum = 0;  // thread = bin; its 32 columns from another start in every lane
#pragma unroll 8
                    for (uint32_t i = 0; i < 32; ++i) {
                        uint32_t &x = columns[tid * 32 + ((i + lane) & 31)];
                        sum += x;
                        x = 0;
                    }
                    if (sum) atomicAdd(p.a.d_hists_or_null + (uint64_t)(is_v ? v_row : k_row) * 256 + tid, sum);
                    __syncthreads();
                }
            }
            t = stop;
        }
    }
}

template <typename T, int kLanes, bool kAdjacent>
static cudaError_t launch_append_lanes(AppendArgs &p, int sms, cudaStream_t s) {
    const uint32_t heads = p.a.q_heads + 2 * p.kv.heads, at_once = 32 / kLanes;
    const uint64_t tokens = p.kv.n_tokens;
    if (p.a.d_hists_or_null) {
        // Counts cost a pass over 32 KB of shared memory per block and request:
        // as many blocks as run at once (half of them keys and half values), of
        // at least a token per warp.  (17.9 us; with two thirds or twice as
        // many blocks 19.7 and 20.1.)
        const uint64_t want = umax64(1, (uint64_t)sms * kCountBlocks / 2);
        p.tokens_per_block = (uint32_t)umax64(kCountWarps, div_up(tokens, want));
        const dim3 grid((uint32_t)umax64(1, div_up(tokens, p.tokens_per_block)), p.a.q_heads ? 3 : 2);
        append_kernel<T, kLanes, kAdjacent, true><<<grid, 32 * kCountWarps, 0, s>>>(p);
        return cudaGetLastError();
    }
    // A warp takes a token's heads in slices.  Each slice looks its token up
    // anew, which costs about as much as four groups of heads, and blocks run
    // in waves of kAppendBlocks per SM: the number of slices with the least
    // waves x (groups + 4).  (Always as many slices as give 24 warps per SM:
    // 4,096 tokens of 48 heads 22.3 us against 21.8.)
    const uint64_t groups = div_up(heads, at_once), blocks = umax64(1, div_up(tokens, kAppendWarps));
    uint64_t best = ~0ull;
    for (uint64_t slices = div_up(groups, 65535); slices <= groups; slices += 1 + slices / 8) {
        const uint64_t each = div_up(groups, slices);
        const uint64_t cost = div_up(blocks * div_up(groups, each), (uint64_t)sms * kAppendBlocks) * (each + 4);
        if (cost < best) {
            best = cost;
            p.slice_heads = (uint32_t)each * at_once;
        }
    }
    p.tokens_per_block = kAppendWarps;
    const dim3 grid((uint32_t)umax64(1, div_up(tokens, kAppendWarps)), (uint32_t)div_up(heads, p.slice_heads));
    append_kernel<T, kLanes, kAdjacent, false><<<grid, 32 * kAppendWarps, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool kAdjacent>
static cudaError_t launch_append_t(AppendArgs &p, int sms, cudaStream_t s) {
    if (p.kv.head_dim <= 64) return launch_append_lanes<T, 8, kAdjacent>(p, sms, s);
    if (p.kv.head_dim <= 128) return launch_append_lanes<T, 16, kAdjacent>(p, sms, s);
    return launch_append_lanes<T, 32, kAdjacent>(p, sms, s);
}

cudaError_t launch_append(const sz_paged_kv &kv, const sz_append_args &a, int32_t *status, int sms, cudaStream_t s) {
    AppendArgs p{};
    p.kv = kv;
    p.a = a;
    p.status = status;
    if (kv.dtype == SZ_BF16)
        return a.interleaved ? launch_append_t<__nv_bfloat16, true>(p, sms, s) : launch_append_t<__nv_bfloat16, false>(p, sms, s);
    return a.interleaved ? launch_append_t<__half, true>(p, sms, s) : launch_append_t<__half, false>(p, sms, s);
}

}  // namespace sz
