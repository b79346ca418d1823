// sz_attention.cu -- softmax attention of new tokens over the paged cache.
//
// Mathematics.  A row's softmax is carried over the keys in one pass with a
// running maximum m, sum l and accumulator o: a key with score s changes them
// to m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') +
// e^(s - m') v; two such triples over different keys join the same way.
// Exponentials are taken base 2 of scores scaled by log2(e).
#include <atomic>
#include <chrono>
#include <type_traits>

#include <unistd.h>

#include "sz_paged.cuh"
#include "sz_tensor.cuh"

namespace sz {

constexpr int kGeneralThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------ any shape
// One block per (new token, query head), any page size and head size: groups
// of kLanes lanes (8 channels each) take keys in turn, each with its own
// running softmax, joined at the end.  What bounds it is the latency of its
// loads and the exchanges between lanes, and every row reads its keys anew:
// it is there for the shapes that the tensor-core kernel does not take.
// (Both on the same calls: one token over 333 keys 28 us, there 12; 5 tokens
// of 16 requests over thousands of keys 1,680 and 45 us; ragged prompts 3,370
// and 63 us.)
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
                const int64_t first = a.window ? max((int64_t)0, (int64_t)q.kv - q.n - a.window + 1) : 0;
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
        // a group whose keys all scored -inf (or without keys) has sums of 0, or
        // NaN where such a key's value was not finite
        const float mg = part[g][kLanes * 8], f = mg == -INFINITY ? 0.0f : exp2f(mg - mm);
        ll += part[g][kLanes * 8 + 1] * f;
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


// ------------------------------------------------------- tensor-core kernel
// Rows of one KV head -- (token, query head) pairs, tokens outermost -- form
// blocks of kM tiles of up to 128; keys come in tiles of up to 128 whole
// pages.  One unit of work is one key tile of one block; the units of all
// requests, heads and blocks in order are dealt in equal runs to the CTAs,
// so a block's keys may be split over several of them (their parts are
// joined afterwards, in order) and a CTA may serve several blocks.
//
// Some warps hold rows, one per thread (softmax); others issue the products,
// the copies of Q and K, and those of V (Shape gives their numbers).  Per row
// tile X and key tile: S_X = Q_X K^T into tensor memory, the softmax threads
// replace S_X by P_X = exp2(c S - c m) in 16 bits in the same columns, O_X +=
// P_X V.  While one row tile's softmax runs, the tensor cores work on the
// other's products (kM = 2) or on the other CTA's of the SM (kM = 1).
//
// What bounds it.  With few rows per request, the reading of the keys and
// values: 64 requests of one token, 735 MB, 129 us in a replayed graph, 5.7
// TB/s (87 % of a copy), 147 us as a call among others; one token over 131,071
// keys 94 us, 5.7 TB/s, and 101.  With long chunks, the products and the
// exponentials and conversions, neither alone: 4,096 tokens over 32,768 keys,
// 32 heads of 128, keep the tensor cores busy for 68 % and the unit that does
// the others for 69 % of the cycles, 1.66 ms in short runs (1,240 TFLOP/s, 74 %
// of the library's matrix products in a burst), 1.91 ms call after call under
// the power cap (1,080 TFLOP/s, 77 % of their sustained rate).  Behind a window
// of 4,096 keys the same two stand at 57 and 58 %; the rest is what does not
// overlap, 2 to 5 us a block: queries, first scores, output.  Ragged prompts
// (64 channels) leave every unit idle for most of the time (tensor cores 20 %,
// exponentials 38 %, memory 8 %): those block ends, key tiles that half of a
// block's rows do not see, and unequal shares (the busiest SM's exponentials
// stand at 53 %).  3 us at the start, in which a CTA finds its share, bound
// short calls (one token over 333 keys: 12 us).
//
// The accumulator is rescaled only when a row's maximum has risen by more
// than 2^8 since the reference that its weights were taken against: until
// then weights up to 2^8 are as exact, and O stays untouched in tensor
// memory.
constexpr uint32_t kTileRows = 128;
constexpr uint32_t kRowBytes = 128;                    // 64 values: one swizzled row
constexpr uint32_t kHalfBytes = kTileRows * kRowBytes;  // 64 channels of a tile
constexpr float kRescaleAt = 8.0f;
// Weights are handed to the products in 16 bits.  FP16 holds none below 2^-25,
// so they are taken 2^7 times larger there, up to 2^15 in all: a key is lost
// below 2^-32 of the largest, and 131,072 lost ones weigh less than a
// sixteenth of half a step.  BF16 has the range of 32 bits.
template <typename T>
__device__ __forceinline__ float reference(float m, float c) {
    return fmaf(m, c, std::is_same<T, __half>::value ? -7.0f : 0.0f);
}
// Blocks up to this many tiles long are not split when there is a CTA for each
// (one token over 333 keys, three tiles: 12.0 us, split and joined 13.4).
constexpr uint32_t kWholeTiles = 6;
constexpr uint64_t kLandingNs = 1000000000;              // after a failed wait, for what is still under way
constexpr uint32_t kMaxTensorSms = 160;                 // workspace bound: CTAs = SMs * CTAs per SM

template <int D, int kM>
struct Shape {
    static constexpr int kTiles = kM, kHalves = D / 64;
    // Rows of a row tile in use.  The products always take 128; with one row
    // tile per CTA only 64 are filled (a few tokens per request), the others
    // read whatever lies behind and their results are not looked at, which
    // leaves room for a third key tile in flight.
    static constexpr uint32_t kRows = kM == 2 ? 128 : 64;
    static constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
    static constexpr int kQueries = D == 64 ? 2 : 1;  // blocks whose queries are in shared memory at a time
    static constexpr int kSlots = kM == 2 ? (D == 128 ? 5 : 10) : (D == 128 ? 3 : 6);
    // Warps.  Which lanes of tensor memory a warp reaches goes by its number
    // modulo 4.  A softmax warp holds 32 rows: with two row tiles all 128
    // columns of a key tile (the row tiles take turns on the tensor cores, and
    // more warps would only share the same arithmetic units), with one row
    // tile half of them, which shortens the chain from tile to tile.
    //   kM = 2: 0..7 softmax, 8 (and 9) products, 9 (or 11) statuses, 10 copies of Q and K, 11 of V
    //   kM = 1: 0, 1 and 4, 5 softmax (4, 5: columns 64 ..), 2 products, 3 and 6 copies, 7 statuses
    static constexpr uint32_t kQuads = kRows / 32;  // warps that hold a row tile's rows
    static constexpr bool kPaired = kM == 1;
    static constexpr uint32_t kMmaWarp = kM == 2 ? 8 : 2, kKeyWarp = kM == 2 ? 10 : 3, kValueWarp = kM == 2 ? 11 : 6;
    // One warp issues the products of both row tiles of 128 channels, which so
    // fall into turns: the products of one run while the other's softmax works
    // (4,096 x 32,768 chunk: 1.66 ms, with a warp each 1.86).  Products of 64
    // channels take half as long as the softmax, and a warp each lets neither
    // wait for the other's weights (ragged prompts: 78 us, with one warp 85).
    static constexpr uint32_t kMmaWarps = kM == 2 && D == 64 ? 2 : 1;
    static constexpr uint32_t kStatusWarp = kM == 1 ? 7 : kMmaWarps == 2 ? kValueWarp : 9;
    static constexpr int kThreads = kM == 2 ? 384 : 256;
    // Registers a thread of the softmax and of the other warps (kM = 2): three
    // warpgroups launched with 168 each, 2 * 208 + 88 = 3 * 168.  The compiler
    // counts with 168 for all: the two-tile kernels spill 62 bytes.
    static constexpr int kManyRegs = 208, kFewRegs = 88;
    static constexpr int kCtasPerSm = kM == 2 ? 1 : 2;
    static constexpr uint32_t kColumns = kM == 2 ? 512 : 256;
    static constexpr uint32_t kQueryHalf = kRows * kRowBytes, kQueryTile = kHalves * kQueryHalf, kQueryBytes = kM * kQueryTile;
    static constexpr uint32_t kData = kQueries * kQueryBytes + kSlots * kTileBytes;
    static constexpr uint32_t kControlBytes = kM == 2 ? 768 : 384 + 2 * 4 * kRows;  // barriers, the CTA's share, exchanged numbers
    static constexpr uint32_t kSmem = kData + kControlBytes;
    // A part of a block: per row tile 4 channels of all rows, the next 4, ...
    // (so that threads that hold a row each write and read side by side),
    // then (m, l) per row.
    static constexpr uint32_t kPartFloats = kM * kRows * (D + 2);
    static __host__ __device__ constexpr uint32_t part_o(uint32_t m_tile, uint32_t chunk, uint32_t row) {
        return ((m_tile * (D / 4) + chunk) * kRows + row) * 4;
    }
    static __host__ __device__ constexpr uint32_t part_ml(uint32_t m_tile, uint32_t row) {
        return kM * kRows * D + (m_tile * kRows + row) * 2;
    }
};

// A block that a CTA began and that goes on in the CTAs after it.
struct SplitRec {
    Request q;
    uint32_t head, block;
    uint32_t last;  // last CTA with a part; 0: none
};

struct TensorArgs {
    sz_paged_kv kv;
    sz_attention_args a;
    float c;               // scale * log2(e), positive
    uint32_t group;        // query heads per KV head
    uint32_t tile_tokens;  // new tokens per row tile
    uint32_t key_tile;     // keys per tile
    uint32_t box_tokens;   // keys per copy
    uint32_t copies;       // copies per key tile and 64 channels
    uint32_t ctas;
    float *parts;          // [ctas][2][kPartFloats]: the part that continues a block, the part that begins one
    SplitRec *rec;         // [ctas]
    unsigned long long *timed_out;  // [2] once a wait of this call ran out: `call`, and the device time
    unsigned long long call;  // this call's tag, 48 bits
    int32_t *status;       // [n_reqs]
    uint64_t wait_limit_ns;
    uint32_t debug_flags;
};

// Whether a wait of this call ran out in another CTA.  Replays of a captured
// call carry one tag, so what an earlier replay left there must go: the join
// clears it, which runs once all CTAs are done; without a join it counts for
// ten seconds (and a wait's limit), far longer than the CTAs of one launch lie
// apart.
constexpr int64_t kRecentNs = 10000000000;
__device__ __forceinline__ bool timed_out(const TensorArgs &p) {
    if (*(volatile unsigned long long *)p.timed_out != p.call) return false;
    __threadfence();
    const int64_t ago = (int64_t)(globaltimer_ns() - *(volatile unsigned long long *)(p.timed_out + 1));
    return ago < kRecentNs || (uint64_t)(ago - kRecentNs) < p.wait_limit_ns;
}

// Visible keys of tokens [first, end) of a request: [*begin, *stop).
__device__ __forceinline__ void key_range(const TensorArgs &p, const Request &q, int32_t first, int32_t end, int32_t *begin,
                                          int32_t *stop) {
    const int32_t p0 = q.kv - q.n + first, p1 = q.kv - q.n + end;  // position of the first, one past the last
    *stop = p.a.causal ? max(0, min(q.kv, p1)) : q.kv;
    *begin = p.a.window ? (int32_t)max((int64_t)0, (int64_t)p0 - p.a.window + 1) : 0;
}

// Key tiles [lo, hi) of block b; at least one, so that rows which see nothing
// are written too.
template <int kM>
__device__ __forceinline__ void block_tiles(const TensorArgs &p, const Request &q, uint32_t b, int32_t *lo, int32_t *hi) {
    const int32_t span = (int32_t)(kM * p.tile_tokens);
    const int32_t first = (int32_t)b * span;
    int32_t begin, stop;
    key_range(p, q, first, min(q.n, first + span), &begin, &stop);
    *lo = begin / (int32_t)p.key_tile;
    *hi = max(*lo + 1, (stop + (int32_t)p.key_tile - 1) / (int32_t)p.key_tile);
}

template <int kM>
__device__ __forceinline__ uint32_t block_count(const TensorArgs &p, const Request &q) {
    const uint32_t span = kM * p.tile_tokens;
    return ((uint32_t)q.n + span - 1) / span;
}

// What a block costs beside its tiles (queries, first scores, output), in
// tiles: the units of a block begin with as many that hold no tile.  Fitted
// to the times of CTAs with blocks of 1 to 40 tiles: 3.4 us beside 1.6 us a
// tile (two row tiles, 64 channels), 5.2 beside 1.8 (128 channels), 0.7 beside
// 2.6 (one row tile, where reading the keys is what takes the time).
template <int D, int kM>
constexpr uint32_t kBlockUnits = kM == 1 ? 0 : D == 64 ? 2 : 3;

// Where a CTA stands in the order of units.
struct Cursor {
    uint32_t r, head, block, off;  // off: tiles of the block done by earlier CTAs
    uint64_t left;                 // units still to do
    bool whole;                    // units are blocks: none is split
    Request q;
};
struct Piece {
    uint32_t r, head, block;
    int32_t t0, t1;     // key tiles
    bool starts, ends;  // holds the block's first, last tile
    Request q;
};

template <int D, int kM>
__device__ __forceinline__ bool next_piece(const TensorArgs &p, Cursor &c, Piece &w) {
    do {
        if (c.left == 0) return false;
        int32_t lo, hi;
        block_tiles<kM>(p, c.q, c.block, &lo, &hi);
        w.r = c.r;
        w.head = c.head;
        w.block = c.block;
        w.q = c.q;
        if (c.whole) {
            w.t0 = lo;
            w.t1 = hi;
            c.left -= 1;
        } else {
            const uint32_t end = c.off + (uint32_t)umin64((uint32_t)(hi - lo) + kBlockUnits<D, kM> - c.off, c.left);
            w.t0 = lo + max((int32_t)(c.off - kBlockUnits<D, kM>), 0);
            w.t1 = lo + max((int32_t)(end - kBlockUnits<D, kM>), 0);
            c.left -= end - c.off;
        }
        w.starts = w.t0 == lo;
        w.ends = w.t1 == hi;
        c.off = 0;
        if (++c.block >= block_count<kM>(p, c.q)) {
            c.block = 0;
            if (++c.head >= p.kv.heads) {
                c.head = 0;
                while (c.left > 0 && ++c.r < p.kv.n_reqs) {
                    c.q = load_request(p.kv, c.r);
                    if (c.q.n > 0) break;
                }
                if (c.r >= p.kv.n_reqs) c.left = 0;
            }
        }
    } while (w.t0 == w.t1);  // a share may end in a block's first units, before its first tile
    return true;
}

// Sums of units, in 32 bits (U) where the call's sizes say that they fit, which
// takes half the instructions: 0.4 us of every call (one token over 333 keys
// 11.8 us, in 64 bits 12.2; both in one kernel, chosen there, gain nothing,
// since it is the fetching of new instructions that takes the time).
template <typename U>
__device__ __forceinline__ U warp_sum(U v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}
template <typename U>
__device__ __forceinline__ U warp_scan(U v, uint32_t lane) {  // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const U y = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= (uint32_t)d) v += y;
    }
    return v;
}

// Quotient of numbers that mostly fit 32 bits.
__device__ __forceinline__ uint32_t divide(uint32_t a, uint32_t b) { return a / b; }
__device__ __forceinline__ uint64_t divide(uint64_t a, uint64_t b) {
    return ((a | b) >> 32) == 0 ? (uint32_t)a / (uint32_t)b : a / b;
}

// Request r (none past the end) and its key tiles per KV head, a request per
// lane of one warp: those of a few blocks are summed by their lane, larger
// ones by all.  `most` grows to the tiles of the longest block, and to
// kDisordered where a request ends before it begins: only rows in order share
// the call's n_tokens, which bounds all sums of units (and the time that this
// takes).
constexpr uint32_t kDisordered = 0xFFFFFFFFu;
template <typename U, int D, int kM>
__device__ U lane_units(const TensorArgs &p, uint32_t r, uint32_t lane, Request &q, uint32_t &most) {
    q.q0 = q.n = q.kv = 0;
    q.status = SZ_OK;
    bool back = false;
    if (r < p.kv.n_reqs) {
        q = load_request(p.kv, r);
        back = __ldg(p.kv.d_q_begin + r + 1) < q.q0;
    }
    if (__any_sync(0xFFFFFFFFu, back)) {
        most = kDisordered;
        return 0;
    }
    const uint32_t blocks = block_count<kM>(p, q);
    U units = 0;
    int32_t lo, hi;
    if (blocks <= 4)
        for (uint32_t b = 0; b < blocks; ++b) {
            block_tiles<kM>(p, q, b, &lo, &hi);
            units += (uint32_t)(hi - lo) + kBlockUnits<D, kM>;
            most = max(most, (uint32_t)(hi - lo));
        }
    uint32_t many = __ballot_sync(0xFFFFFFFFu, blocks > 4);
    while (many) {
        const int src = __ffs(many) - 1;
        many &= many - 1;
        Request x;
        x.q0 = __shfl_sync(0xFFFFFFFFu, q.q0, src);
        x.n = __shfl_sync(0xFFFFFFFFu, q.n, src);
        x.kv = __shfl_sync(0xFFFFFFFFu, q.kv, src);
        const uint32_t n = block_count<kM>(p, x);
        U sum = 0;
        for (uint32_t b = lane; b < n; b += 32) {
            block_tiles<kM>(p, x, b, &lo, &hi);
            sum += (uint32_t)(hi - lo) + kBlockUnits<D, kM>;
            most = max(most, (uint32_t)(hi - lo));
        }
        sum = warp_sum(sum);
        if ((int)lane == src) units = sum;
    }
    return units;
}

struct PlanShared {
    uint64_t total;
    uint64_t first, left;  // this CTA's units
    uint32_t used;         // CTAs with work
    uint32_t r, head, block, off;
    bool whole;
    Request q;
};

// What the search for it exchanges between warps.
struct PlanScratch {
    uint64_t units[12], blocks[12];
    uint32_t most[12];
};

// This CTA's share of the units, found by all of its threads.
template <typename U, int D, int kM>
__device__ void find_share(const TensorArgs &p, PlanShared &s, PlanScratch &x) {
    constexpr uint32_t kW = Shape<D, kM>::kThreads / 32;
    const uint32_t lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const uint32_t rounds = (p.kv.n_reqs + 32 * kW - 1) / (32 * kW);
    U mine = 0, per_head = 0, blocks = 0;
    uint32_t most = 0;
    Request q;
    for (uint32_t i = 0; i < rounds; ++i) {
        per_head = lane_units<U, D, kM>(p, (wid * rounds + i) * 32 + lane, lane, q, most);
        mine += per_head;
        blocks += block_count<kM>(p, q);
    }
    mine = warp_sum(mine) * p.kv.heads;
    blocks = warp_sum(blocks) * p.kv.heads;
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) {
        x.units[wid] = mine;
        x.blocks[wid] = blocks;
        x.most[wid] = most;
    }
    __syncthreads();
    U total = 0, before = 0, total_blocks = 0, before_blocks = 0;
    for (uint32_t w = 0; w < kW; ++w) {
        if (w < wid) before += (U)x.units[w], before_blocks += (U)x.blocks[w];
        total += (U)x.units[w];
        total_blocks += (U)x.blocks[w];
        most = max(most, x.most[w]);
    }
    // A few short blocks: one CTA each, which costs less than joining parts.
    const bool whole = total_blocks <= p.ctas && most <= kWholeTiles;
    if (whole) total = total_blocks, before = before_blocks, mine = blocks;
    if (most == kDisordered) total = 0;  // the requests overlap: nothing is done, and the statuses say so
    // Every CTA that works has at least one unit, so that the parts of a block
    // are those of consecutive CTAs.
    const U used = total < p.ctas ? (total > 0 ? total : 1) : p.ctas;
    const bool works = blockIdx.x < used;
    const U u0 = works ? divide(blockIdx.x * total, used) : 0, u1 = works ? divide((blockIdx.x + 1) * total, used) : 0;
    if (threadIdx.x == 0) {
        s.left = 0;
        s.first = u0;
        s.total = total;
        s.used = (uint32_t)used;
        s.whole = whole;
    }
    __syncthreads();
    if (u1 > u0 && u0 >= before && u0 < before + mine) {  // one warp
        U rem = u0 - before;
        for (uint32_t i = 0; i < rounds; ++i) {
            const uint32_t r0 = (wid * rounds + i) * 32;
            if (rounds > 1) per_head = lane_units<U, D, kM>(p, r0 + lane, lane, q, most);
            const U units = whole ? block_count<kM>(p, q) : per_head;
            const U end = warp_scan<U>(units * p.kv.heads, lane);
            const uint32_t hit = __ballot_sync(0xFFFFFFFFu, rem < end);
            if (hit == 0) {
                rem -= __shfl_sync(0xFFFFFFFFu, end, 31);
                continue;
            }
            const int src = __ffs(hit) - 1;
            const U w = __shfl_sync(0xFFFFFFFFu, units, src);
            rem -= __shfl_sync(0xFFFFFFFFu, end - units * p.kv.heads, src);
            const uint32_t head = (uint32_t)divide(rem, w);
            rem -= head * w;
            Request own;
            own.q0 = __shfl_sync(0xFFFFFFFFu, q.q0, src);
            own.n = __shfl_sync(0xFFFFFFFFu, q.n, src);
            own.kv = __shfl_sync(0xFFFFFFFFu, q.kv, src);
            own.status = SZ_OK;
            for (uint32_t b0 = 0; b0 < block_count<kM>(p, own); b0 += 32) {
                U n = 0;
                if (b0 + lane < block_count<kM>(p, own)) {
                    int32_t lo, hi;
                    block_tiles<kM>(p, own, b0 + lane, &lo, &hi);
                    n = whole ? 1u : (uint32_t)(hi - lo) + kBlockUnits<D, kM>;
                }
                const U stop = warp_scan<U>(n, lane);
                const uint32_t here = __ballot_sync(0xFFFFFFFFu, rem < stop);
                if (here == 0) {
                    rem -= __shfl_sync(0xFFFFFFFFu, stop, 31);
                    continue;
                }
                const int at = __ffs(here) - 1;
                rem -= __shfl_sync(0xFFFFFFFFu, stop - n, at);
                if (lane == 0) {
                    s.r = r0 + (uint32_t)src;
                    s.head = head;
                    s.block = b0 + (uint32_t)at;
                    s.off = (uint32_t)rem;
                    s.q = own;
                    s.left = u1 - u0;
                }
                break;
            }
            break;
        }
    }
    __syncthreads();
}

// The CTA that has unit u.
__device__ __forceinline__ uint32_t cta_of(const PlanShared &s, uint64_t u) {
    return (uint32_t)divide((u + 1) * s.used - 1, s.total);
}

// What the roles of a CTA tell one another beside its barriers: that a wait
// ran out, and how many warps sum rows again (mend_rows), which may take longer
// than any wait should.
struct Watch {
    uint32_t failed, busy;
};

// Wait for a phase; false when the limit of device time ran out here (since
// the last look that found no warp busy) or elsewhere in the CTA.
__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, volatile Watch *watch, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (watch->failed) return false;
        const uint64_t now = globaltimer_ns();
        if (watch->busy) t0 = now;
        if (now - t0 > limit_ns) {
            watch->failed = 1u;
            return false;
        }
    }
    return true;
}
// The roles whose accesses stay in bounds whatever the data go on after a
// failure, which ends all further waits at once; but the products' warp hands
// nothing back that it has not seen land, so that no copy is issued over one
// under way.  A copying warp asks this, for all of its lanes, and stops.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile Watch *watch, uint64_t limit_ns) {
    return __all_sync(0xFFFFFFFFu, wait_or_fail(bar, parity, watch, limit_ns)) != 0;
}

// Columns outside [from, to) of a row's scores become -inf.
template <int N>
__device__ __forceinline__ void hide(uint32_t (&s)[N], int32_t from, int32_t to) {
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < from || j >= to) s[j] = 0xFF800000u;
}

// Barriers of the two warps that hold the same rows; one also tells whether
// any of their threads has `x`.
__device__ __forceinline__ void pair_sync(uint32_t id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_any(uint32_t id, bool x) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "bar.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(id), "r"(x ? 1u : 0u)
        : "memory");
    return any != 0;
}

// Whether any row of the warp, or of the pair, asks for another reference.
template <bool kPaired>
__device__ __forceinline__ bool asks(uint32_t pair, bool x) {
    if constexpr (kPaired) return pair_any(pair, x);
    return __any_sync(0xFFFFFFFFu, x) != 0;
}

// Which of two 16-bit values are infinite or NaN: bits 0 and 16.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t pair) {
    constexpr uint32_t kExponent = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
    return ((pair & kExponent) == kExponent ? 1u : 0u) | ((pair >> 16 & kExponent) == kExponent ? 0x10000u : 0u);
}

// Rows (one per lane, where `odd`) whose accumulator holds a NaN while their
// sum does not: somewhere a weight met a value that is not finite.  It was the
// weight of a key that the row sees, whose infinity or NaN belongs in the
// result (also where the weight was so small that it became 0 in 16 bits, and
// 0 times infinity NaN), or the 0 of a hidden key, whose value does not.  So
// the keys that the row sees, [from, to) of those in hand, are looked through
// for such values, a key per lane at a time, and what they come to replaces
// the accumulator's NaNs: an infinity where only values of its sign were met,
// NaN where both were, or a NaN, or a key of weight exactly 0.  A NaN that met
// none came from a hidden key: that channel is summed again, 2^(c s_j - ref) v_j
// over the keys that the row sees.  `o_at` holds channels [c0, c0 + kOwn).
// Both are bound by the latency of a key's loads.  A chunk of 4,096 tokens over
// 32,768 keys (32 heads of 128, 1.65 ms) takes no longer where all rows see an
// infinity, 94 ms where a channel is infinite in every key, 160 ms where the
// last token's value is NaN and the two blocks per KV head that must not see it
// are summed again.
template <typename T, int D, int kOwn>
__device__ __noinline__ void mend_rows(const TensorArgs *p, Watch *watch, uint32_t r, uint32_t kv_head, const uint16_t *q, bool odd, int32_t from,
                                       int32_t to, float ref, uint32_t o_at, uint32_t c0) {
    const sz_paged_kv &kv = p->kv;
    const uint32_t lane = threadIdx.x & 31;
    if (lane == 0) atomicAdd(&watch->busy, 1u);
    const uint16_t *const keys = (const uint16_t *)kv.d_k + kv_head * kv.k_stride[1];
    const uint16_t *values = (const uint16_t *)kv.d_v + kv_head * kv.v_stride[1] + c0;
    bool q_infinite = false;
    if (odd)
#pragma unroll 1
        for (int i = 0; i < D; i += 2) q_infinite |= not_finite<T>(*(const uint32_t *)(q + i)) != 0;
#pragma unroll 1
    for (int w = 0; w < kOwn / 32; ++w, o_at += 32, values += 32) {  // 32 channels at a time, a bit each
        uint32_t a[32];
        tmem_ld32(o_at, a);
        tmem_wait_ld();
        uint32_t nan = 0, up = 0, down = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (odd && __uint_as_float(a[i]) != __uint_as_float(a[i])) nan |= 1u << i;
        bool open = __any_sync(0xFFFFFFFFu, nan != 0) != 0;  // some row's NaN is not explained for good
        if (!open) continue;
        const int32_t end = __reduce_max_sync(0xFFFFFFFFu, nan ? to : 0);
#pragma unroll 1
        for (int32_t j0 = __reduce_min_sync(0xFFFFFFFFu, nan ? from : 0x7FFFFFFF); open && j0 < end; j0 += 32) {
            const int32_t j = j0 + (int32_t)lane;
            const int32_t page = j < end ? page_of(kv, r, (uint32_t)j / kv.page_tokens) : -1;
            const uint32_t slot = (uint32_t)j % kv.page_tokens;
            uint32_t found = 0;
            if (page >= 0) {
                const uint16_t *const v = values + (uint64_t)page * kv.v_stride[0] + slot * kv.v_stride[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 y = *(const uint4 *)(v + i * 8);
                    found |= not_finite<T>(y.x) | not_finite<T>(y.y) | not_finite<T>(y.z) | not_finite<T>(y.w);
                }
            }
            uint32_t hits = __ballot_sync(0xFFFFFFFFu, found != 0);
#pragma unroll 1
            while (open && hits) {
                const int src = __ffs(hits) - 1;
                hits &= hits - 1;
                const uint64_t key_page = (uint64_t)__shfl_sync(0xFFFFFFFFu, page, src), key_slot = __shfl_sync(0xFFFFFFFFu, slot, src);
                const uint32_t bits = (values + key_page * kv.v_stride[0] + key_slot * kv.v_stride[2])[lane];
                const bool sees = odd && j0 + src >= from && j0 + src < to;
                // weight 0: a score of -inf, which finite numbers come to by
                // overflow at most
                const uint16_t *const k = keys + key_page * kv.k_stride[0] + key_slot * kv.k_stride[2];
                bool infinite = q_infinite;
                for (uint32_t i = 2 * lane; i < D; i += 64) infinite |= not_finite<T>(*(const uint32_t *)(k + i)) != 0;
                bool nothing = false;
                if (__any_sync(0xFFFFFFFFu, infinite) && sees) {
                    float s = 0.0f;
#pragma unroll 1
                    for (int i = 0; i < D; i += 8) {
                        float x[8], y[8];
                        widen8<T>(*(const uint4 *)(q + i), x);
                        widen8<T>(*(const uint4 *)(k + i), y);
#pragma unroll
                        for (int e = 0; e < 8; ++e) s += x[e] * y[e];
                    }
                    nothing = s == -INFINITY;
                }
                const float y = Half2<T>::widen(bits).x;
                const bool any = not_finite<T>(bits) != 0;
                const uint32_t up1 = __ballot_sync(0xFFFFFFFFu, any && !(y < 0.0f)), down1 = __ballot_sync(0xFFFFFFFFu, any && !(y > 0.0f));
                if (sees) {
                    up |= nothing ? up1 | down1 : up1;
                    down |= nothing ? up1 | down1 : down1;
                }
                open = __any_sync(0xFFFFFFFFu, (nan & ~(up & down)) != 0) != 0;
            }
        }
        const uint32_t lost = nan & ~(up | down);
        float o[32] = {};
        const int32_t end1 = __reduce_max_sync(0xFFFFFFFFu, lost ? to : 0);
#pragma unroll 1
        for (int32_t j0 = __reduce_min_sync(0xFFFFFFFFu, lost ? from : 0x7FFFFFFF); j0 < end1; j0 += 32) {
            const int32_t j = j0 + (int32_t)lane;
            const int32_t page = j < end1 ? page_of(kv, r, (uint32_t)j / kv.page_tokens) : -1;
            const uint32_t here = __ballot_sync(0xFFFFFFFFu, page >= 0);
            // keys without a page: the pool's first, with weight 0
            const uint64_t page1 = page >= 0 ? (uint32_t)page : 0, slot = page >= 0 ? (uint32_t)j % kv.page_tokens : 0;
            const uint64_t k_at = (uint64_t)(keys + page1 * kv.k_stride[0] + slot * kv.k_stride[2]);
            const uint64_t v_at = (uint64_t)(values + page1 * kv.v_stride[0] + slot * kv.v_stride[2]);
#pragma unroll 1
            for (int t = 0; t < 32; t += 2) {
                // two keys at a time, which share the loads of q; those after next are on their way to the first cache
                const int ahead = (t + 4 + (int)(lane / 16)) & 31;
                const uint64_t k_ahead = __shfl_sync(0xFFFFFFFFu, k_at, ahead), v_ahead = __shfl_sync(0xFFFFFFFFu, v_at, ahead);
                asm volatile("prefetch.global.L1 [%0];" ::"l"(k_ahead + lane % 16 * (D / 8)));
                asm volatile("prefetch.global.L1 [%0];" ::"l"(v_ahead + lane % 16 * 4));
                const uint16_t *const k0 = (const uint16_t *)__shfl_sync(0xFFFFFFFFu, k_at, t), *const k1 = (const uint16_t *)__shfl_sync(0xFFFFFFFFu, k_at, t + 1);
                const uint16_t *const v0 = (const uint16_t *)__shfl_sync(0xFFFFFFFFu, v_at, t), *const v1 = (const uint16_t *)__shfl_sync(0xFFFFFFFFu, v_at, t + 1);
                const bool sees0 = lost && j0 + t >= from && j0 + t < to && (here >> t & 1u), sees1 = lost && j0 + t + 1 >= from && j0 + t + 1 < to && (here >> t & 2u);
                if (!sees0 && !sees1) continue;
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 1
                for (int i = 0; i < D; i += 8) {
                    float x[8], y[8];
                    widen8<T>(*(const uint4 *)(q + i), x);
                    widen8<T>(*(const uint4 *)(k0 + i), y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s0 += x[e] * y[e];
                    widen8<T>(*(const uint4 *)(k1 + i), y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s1 += x[e] * y[e];
                }
                const float e0 = exp2f(fmaf(s0, p->c, -ref)), e1 = exp2f(fmaf(s1, p->c, -ref));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y[8];
                    widen8<T>(*(const uint4 *)(v0 + i * 8), y);
                    if (sees0)
#pragma unroll
                        for (int c = 0; c < 8; ++c) o[i * 8 + c] += e0 * y[c];
                    widen8<T>(*(const uint4 *)(v1 + i * 8), y);
                    if (sees1)
#pragma unroll
                        for (int c = 0; c < 8; ++c) o[i * 8 + c] += e1 * y[c];
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t b[16];
            tmem_ld16(o_at + h * 16, b);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t bit = 1u << (h * 16 + i);
                if (lost & bit) b[i] = __float_as_uint(o[h * 16 + i]);
                if (nan & (up ^ down) & bit) b[i] = up & bit ? 0x7F800000u : 0xFF800000u;
            }
            tmem_st16(o_at + h * 16, b);
        }
    }
    tmem_wait_st();
    if (lane == 0) atomicSub(&watch->busy, 1u);
    __syncwarp();
}

struct Bars {
    uint64_t full[10], empty[10];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2][2], pv_done[2];
    uint64_t drain[2];
};

template <int D, int kM>
struct Control {  // behind the tiles in shared memory
    Bars bars;
    PlanShared plan;
    uint32_t tmem;
    Watch watch;
    uint32_t issued[2], queries;  // uses of the ring that K's and V's copies stand behind, blocks whose queries were copied
    union {
        PlanScratch scratch;
        float swap[2][Shape<D, kM>::kPaired ? Shape<D, kM>::kRows : 1];  // between the two halves of a row: maxima, sums
    };
};

template <typename T, int D, int kM, typename U>
__global__ void __launch_bounds__(Shape<D, kM>::kThreads, Shape<D, kM>::kCtasPerSm)
attention_kernel(const __grid_constant__ TensorArgs p, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using S = Shape<D, kM>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kScoreWord = mma_word(kBf16, 128, false);
    constexpr uint32_t kOutWord = mma_word(kBf16, D, true);
    extern __shared__ __align__(1024) uint8_t raw[];
    using Control = Control<D, kM>;
    static_assert(sizeof(Control) <= S::kControlBytes, "control block");
    Control &control = *reinterpret_cast<Control *>(raw + S::kData);
    Bars &bars = control.bars;
    PlanShared &plan = control.plan;
    const volatile uint32_t &failed = control.watch.failed;
    // what is the same for a whole warp is passed through a shuffle, so that
    // the compiler keeps it in uniform registers, where the tensor
    // instructions want their operands
    const uint32_t tid = threadIdx.x, wid = same(tid >> 5), lane = tid & 31;
    const uint32_t smem0 = smem_u32(raw);
    const uint32_t ring0 = smem0 + S::kQueries * S::kQueryBytes;
    constexpr uint32_t kMmaWarp = S::kMmaWarp;
    const bool softmax = kM == 2 ? wid < 8 : (wid & 3) < 2 && wid < 6;

    if (wid == kMmaWarp) tmem_alloc(&control.tmem, S::kColumns);
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], S::kMmaWarps);
        }
        for (int i = 0; i < S::kQueries; ++i) {
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], S::kMmaWarps);
        }
        for (int x = 0; x < kM; ++x) {
            mbar_init(&bars.s_full[x], 1);
            mbar_init(&bars.p_full[x][0], S::kQuads);
            mbar_init(&bars.p_full[x][1], S::kQuads);
            mbar_init(&bars.pv_done[x], 1);
        }
        mbar_init(&bars.drain[0], 1);
        mbar_init(&bars.drain[1], 1);
        fence_mbar_init();
        control.watch.failed = control.watch.busy = 0;
    }
    if (wid == S::kKeyWarp && lane == 0) {
        prefetch_map(&q_map);
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    }
    // Rows of a tile that no copy writes (pages that do not divide 128) hold
    // zeros from here on: their weights are 0, and so must be what they meet.
    if (p.key_tile < kTileRows)
        for (uint32_t i = tid; i < S::kSlots * S::kHalves * (kTileRows - p.key_tile) * 8; i += S::kThreads) {
            const uint32_t piece = i % 8, row = p.key_tile + i / 8 % (kTileRows - p.key_tile), half = i / 8 / (kTileRows - p.key_tile);
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(ring0 + half * kHalfBytes + row * kRowBytes + piece * 16), "r"(0) : "memory");
        }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    find_share<U, D, kM>(p, plan, control.scratch);  // synchronises the block
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (p.rec) allow_dependents();  // the join, which waits; another kernel might read `out` too early
    const uint32_t tmem = same(control.tmem);
    Cursor cur;
    cur.r = plan.r;
    cur.head = plan.head;
    cur.block = plan.block;
    cur.off = plan.off;
    cur.left = plan.left;
    cur.whole = plan.whole;
    cur.q = plan.q;
    volatile Watch *const watch = &control.watch;
    const uint64_t limit = p.wait_limit_ns;
    Piece w;
    if (!softmax) {
        if constexpr (kM == 2) give_registers<S::kFewRegs>();
        if (wid == S::kKeyWarp || wid == S::kValueWarp) {
        // ------------------------------------- copies: Q and K, or V
        const bool one = elect_one();
        const uint32_t is_v = wid == S::kValueWarp ? 1u : 0u;
        const CUtensorMap *const map = is_v ? &v_map : &k_map;
        const bool silent = is_v && (p.debug_flags & kDebugNoSignal) != 0;  // a test of waits that run out
        const uint32_t tile_bytes = p.key_tile * S::kHalves * kRowBytes;
        const uint32_t copy_bytes = p.box_tokens * kRowBytes;
        uint32_t use = is_v, pieces = 0;  // of the ring (K even, V odd), pieces begun
        bool ok = true;
        SplitRec rec;
        rec.last = 0;
        while (ok && next_piece<D, kM>(p, cur, w)) {
            if (w.starts && !w.ends) {
                int32_t lo, hi;
                block_tiles<kM>(p, w.q, w.block, &lo, &hi);
                rec.q = w.q;
                rec.head = w.head;
                rec.block = w.block;
                // of the units left, those of this block's other tiles come last
                rec.last = cta_of(plan, plan.first + plan.left + (uint32_t)(hi - w.t1) - 1);
            }
            const uint32_t first = w.block * kM * p.tile_tokens;
            const uint32_t tokens = umin32((uint32_t)w.q.n - first, kM * p.tile_tokens);
            const uint32_t tiles = kM == 1 || tokens <= p.tile_tokens ? 1u : 2u;
            const uint32_t head = same(w.head);
            if (!is_v) {
                const uint32_t buf = pieces % S::kQueries;
                if (!(ok = warp_wait(&bars.q_empty[buf], (pieces / S::kQueries & 1) ^ 1, watch, limit))) break;
                ++pieces;
                if (one) {
                    const uint32_t rows = p.tile_tokens * p.group;
                    mbar_arrive_expect_tx(&bars.q_full[buf], tiles * rows * S::kHalves * kRowBytes);
                    for (uint32_t x = 0; x < tiles; ++x)
#pragma unroll
                        for (uint32_t hf = 0; hf < (uint32_t)S::kHalves; ++hf)
                            tma_load_3d(smem0 + buf * S::kQueryBytes + x * S::kQueryTile + hf * S::kQueryHalf, &q_map, (int)(hf * 64), (int)(head * p.group),
                                        (int)((uint32_t)w.q.q0 + first + x * p.tile_tokens), smem_u32(&bars.q_full[buf]));
                }
                __syncwarp();
            }
            int32_t begin, stop;
            key_range(p, w.q, (int32_t)first, (int32_t)(first + tokens), &begin, &stop);
            const int32_t page_lo = begin / (int32_t)p.kv.page_tokens;
            const int32_t page_hi = (w.q.kv + (int32_t)p.kv.page_tokens - 1) / (int32_t)p.kv.page_tokens;
            // Pages behind the last token, before the window or outside the
            // pool are copied from behind the pool's end: zeros.
            auto page_at = [&](int32_t t) -> int32_t {
                const int32_t i = t * (int32_t)p.key_tile / (int32_t)p.kv.page_tokens + (int32_t)lane;
                int32_t page = -1;
                if (lane < p.copies && i >= page_lo && i < page_hi) page = page_of(p.kv, w.r, (uint32_t)i);
                return page < 0 ? (int32_t)p.kv.n_pages : page;
            };
            int32_t page = page_at(w.t0);
            const int32_t t_end = (int32_t)same((uint32_t)w.t1);
            for (int32_t t = (int32_t)same((uint32_t)w.t0); t < t_end; ++t, use += 2) {
                const int32_t token = p.box_tokens < p.kv.page_tokens ? t * (int32_t)p.key_tile % (int32_t)p.kv.page_tokens : 0;
                const uint32_t slot = use % S::kSlots, phase = use / S::kSlots & 1;
                if (!(ok = warp_wait(&bars.empty[slot], phase ^ 1, watch, limit))) break;
                const uint32_t bar = smem_u32(&bars.full[slot]);
                if (one) mbar_arrive_expect_tx(&bars.full[slot], tile_bytes);
                uint32_t dst = ring0 + slot * S::kTileBytes;
                for (uint32_t i = 0; i < p.copies; ++i, dst += copy_bytes) {
                    const int32_t from = (int32_t)__shfl_sync(0xFFFFFFFFu, page, i);
                    if (one && !silent) {
#pragma unroll
                        for (uint32_t hf = 0; hf < (uint32_t)S::kHalves; ++hf)
                            tma_load_4d(dst + hf * kHalfBytes, map, (int)(hf * 64), token, (int)head, from, bar);
                    }
                }
                __syncwarp();
                if (t + 1 < t_end) page = page_at(t + 1);
            }
        }
        if (p.rec && is_v && lane == 0) p.rec[blockIdx.x] = rec;
        if (lane == 0) {
            control.issued[is_v] = use;
            if (!is_v) control.queries = pieces;
        }
        } else if (wid >= kMmaWarp && wid < kMmaWarp + S::kMmaWarps) {
        // ---------------------------------------------------------- products
        const bool one = elect_one();
        const uint32_t q_lo = desc_lo(smem0, 16), k_lo = desc_lo(ring0, 16), v_lo = desc_lo(ring0, kHalfBytes);
        uint32_t done = 0, done2 = 0;  // key tiles of this warp's row tile, or of the first and the second
        uint32_t slot = 0, phase = 0;  // of the ring, at the next K or V
        auto pass = [&] {              // to the next of the ring
            if (++slot == S::kSlots) slot = 0, phase ^= 1;
        };
        const uint32_t mine = wid - kMmaWarp;
        bool landed = true;            // every copy waited for so far
        auto each = [&](auto f) {  // row tile of this warp's
            if constexpr (S::kMmaWarps == 2) {
                f(mine);
            } else {
#pragma unroll
                for (uint32_t m = 0; m < kM; ++m) f(m);
            }
        };
        for (uint32_t piece = 0; same(failed) == 0; ++piece) {
            if (same(next_piece<D, kM>(p, cur, w) ? 1u : 0u) == 0) break;
            const int32_t t_begin = (int32_t)same((uint32_t)w.t0), t_end = (int32_t)same((uint32_t)w.t1), kv = (int32_t)same((uint32_t)w.q.kv);
            const uint32_t tiles = same(kM == 1 || (uint32_t)w.q.n - w.block * kM * p.tile_tokens <= p.tile_tokens ? 1u : 2u);  // row tiles in use
            const uint32_t buf = piece % S::kQueries;
            auto score = [&](uint32_t m) {  // S_m = Q_m K^T, K at `slot`
                const uint32_t qa = q_lo + buf * (S::kQueryBytes >> 4) + m * (S::kQueryTile >> 4), b = k_lo + slot * (S::kTileBytes >> 4);
                if (one) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t half = (uint32_t)(i / 4), off = (uint32_t)(i % 4) * 32 >> 4;
                        mma_smem(tmem + m * 128, full_desc(qa + half * (S::kQueryHalf >> 4) + off), full_desc(b + half * (kHalfBytes >> 4) + off), kScoreWord, i > 0);
                    }
                    mma_commit(&bars.s_full[m]);
                }
                __syncwarp();
            };
            landed &= wait_or_fail(&bars.q_full[buf], piece / S::kQueries & 1, watch, limit);
            landed &= wait_or_fail(&bars.full[slot], phase, watch, limit);
            tc_fence_after();
            each([&](uint32_t m) {
                if (m < tiles) score(m);
            });
            if (one && landed) mma_commit(&bars.empty[slot]);
            pass();
            for (int32_t t = t_begin; t < t_end; ++t) {
                const uint32_t v_slot = slot;
                const bool more = t + 1 < t_end;
                landed &= wait_or_fail(&bars.full[slot], phase, watch, limit);
                pass();
                if (more)  // the next K now, so that nothing is waited for between the products
                    landed &= wait_or_fail(&bars.full[slot], phase, watch, limit);
                else if (one && landed)
                    mma_commit(&bars.q_empty[buf]);
                // keys behind the last token in this tile's last page: their
                // weights are 0, so their values must be finite
                const int32_t z0 = kv - t * (int32_t)p.key_tile;
                if (z0 > 0 && z0 < (int32_t)p.key_tile) {
                    const int32_t page = (int32_t)p.kv.page_tokens;
                    const int32_t z1 = (int32_t)min((int64_t)p.key_tile, ((int64_t)kv + page - 1) / page * page - (int64_t)t * p.key_tile);
                    const uint32_t vb = ring0 + v_slot * S::kTileBytes;
                    for (int32_t i = (int32_t)lane; i < (z1 - z0) * S::kHalves * 8; i += 32) {
                        const uint32_t chunk = i % 8, half = i / 8 % S::kHalves, row = (uint32_t)(z0 + i / 8 / S::kHalves);
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vb + half * kHalfBytes + row * kRowBytes + chunk * 16), "r"(0)
                                     : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                const uint32_t vb = v_lo + v_slot * (S::kTileBytes >> 4);
                each([&](uint32_t m) {
                    if (m < tiles) {
#pragma unroll
                        for (uint32_t part = 0; part < 2; ++part) {  // the weights of 64 keys each
                            wait_or_fail(&bars.p_full[m][part], (S::kMmaWarps == 1 && m == 1 ? done2 : done) & 1, watch, limit);
                            tc_fence_after();
                            if (one) {
#pragma unroll
                                for (uint32_t i = 0; i < 4; ++i)
                                    mma_tmem(tmem + kM * 128 + m * D, tmem + m * 128 + part * 64 + i * 8, full_desc(vb + (part * 4 + i) * (16 * kRowBytes >> 4)),
                                             kOutWord, (t > t_begin || part + i > 0) ? 1u : 0u);
                                if (part == 1) mma_commit(&bars.pv_done[m]);
                            }
                            __syncwarp();
                        }
                    }
                    if (one && landed && (S::kMmaWarps == 2 || m + 1 == kM)) mma_commit(&bars.empty[v_slot]);
                    if (more && m < tiles) score(m);
                });
                if (S::kMmaWarps == 2) done += mine < tiles ? 1 : 0; else ++done, done2 += tiles > 1 ? 1 : 0;
                if (more && one && landed) mma_commit(&bars.empty[slot]);
                if (more) pass();
            }
        }
        }
    } else {
        // ----------------------------------------------------------- softmax

        if constexpr (kM == 2) take_registers<S::kManyRegs>();
        constexpr uint32_t kParts = S::kPaired ? 1 : 2;    // of 64 columns, per warp
        constexpr uint32_t kOwn = S::kPaired ? D / 2 : D;  // channels that a warp rescales and writes
        const uint32_t m_tile = kM == 2 ? wid / 4 : 0, half = S::kPaired ? wid / 4 : 0, quad = wid & 3;
        const uint32_t row = quad * 32 + lane;
        const uint32_t lanes = quad * 32;  // of tensor memory
        const uint32_t pair = 1 + quad;    // barrier of the two warps that share rows
        const uint32_t s_at = tmem + (lanes << 16) + m_tile * 128 + half * 64;
        const uint32_t o_at = tmem + (lanes << 16) + kM * 128 + m_tile * D + half * kOwn;
        float *const swap_mine = &control.swap[half][S::kPaired ? row : 0], *const swap_other = &control.swap[half ^ 1][S::kPaired ? row : 0];
        const uint32_t my_token = row / p.group, my_head = row % p.group;
        uint32_t n = 0;  // tiles done by this row tile
        while (next_piece<D, kM>(p, cur, w)) {
            const uint32_t first = (w.block * kM + m_tile) * p.tile_tokens;
            if ((uint32_t)w.q.n <= first) continue;
            const uint32_t rows = umin32((uint32_t)w.q.n - first, p.tile_tokens) * p.group;
            const bool warp_live = lanes < rows;
            int32_t begin, stop;
            key_range(p, w.q, (int32_t)(first + my_token), (int32_t)(first + my_token) + 1, &begin, &stop);
            float m = -INFINITY;             // reference of the weights
            uint64_t sum = pack2(0.0f, 0.0f);  // of this half's weights, in two parts
            for (int32_t t = w.t0; t < w.t1; ++t, ++n) {
                wait_or_fail(&bars.s_full[m_tile], n & 1, watch, limit);
                tc_fence_after();
                if (warp_live) {
                    // this row's visible columns; all of them in most tiles
                    const int32_t k0 = t * (int32_t)p.key_tile;
                    const int32_t from = begin - k0 - (int32_t)half * 64, to = min(stop - k0, (int32_t)p.key_tile) - (int32_t)half * 64;
                    const bool masked = __any_sync(0xFFFFFFFFu, from > 0 || to < (int32_t)kParts * 64) != 0;
                    uint32_t s[kParts][64];
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    tmem_ld64(s_at, s[0]);
                    tmem_wait_ld();
                    if constexpr (kParts == 2) tmem_ld64(s_at + 64, s[1]);
#pragma unroll
                    for (uint32_t part = 0; part < kParts; ++part) {
                        if (part) tmem_wait_ld();
                        if (masked) hide(s[part], from - (int32_t)part * 64, to - (int32_t)part * 64);
#pragma unroll
                        for (int j = 0; j < 64; j += 8)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                top[i] = max3(top[i], __uint_as_float(s[part][j + 2 * i]), __uint_as_float(s[part][j + 2 * i + 1]));
                    }
                    float high = fmaxf(max3(top[0], top[1], top[2]), top[3]);
                    // A row has one reference: it moves at first and then
                    // rarely, for both of a pair of warps when either asks.
                    const bool begins = t == w.t0;
                    if (begins || asks<S::kPaired>(pair, (high - m) * p.c > kRescaleAt)) {
                        if constexpr (S::kPaired) {
                            *swap_mine = high;
                            pair_sync(pair);
                            high = fmaxf(high, *swap_other);
                        }
                        if (begins) {
                            m = high;
                        } else {
                            // the accumulator as of the tile before
                            wait_or_fail(&bars.pv_done[m_tile], (n - 1) & 1, watch, limit);
                            tc_fence_after();
                            const bool rise = (high - m) * p.c > kRescaleAt;
                            const float f = rise ? exp2_fast((m - high) * p.c) : 1.0f;
                            if (rise) m = high;
                            sum = mul2(sum, pack2(f, f));
#pragma unroll 1
                            for (uint32_t i = 0; i < kOwn / 16; ++i) {
                                uint32_t o[16];
                                tmem_ld16(o_at + i * 16, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st16(o_at + i * 16, o);
                            }
                            tmem_wait_st();
                            tc_fence_before();
                            if constexpr (S::kPaired) pair_sync(pair);  // the other's channels too, before any weight is handed over
                        }
                    }
                    const float ref = m == -INFINITY ? 0.0f : reference<T>(m, p.c);
                    const uint64_t c2 = pack2(p.c, p.c), ref2 = pack2(-ref, -ref);
                    // summed by tile first: a small weight beside a large running
                    // sum would be lost, 128 of them less so
                    uint64_t sum0 = pack2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
                    for (uint32_t i = 0; i < kParts * 2; ++i) {  // weights of 64 columns take the first 32 of them
                        uint32_t w16[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int at = (int)(i & 1) * 32 + 2 * j;
                            const uint64_t x = fma2(pack2(__uint_as_float(s[i / 2][at]), __uint_as_float(s[i / 2][at + 1])), c2, ref2);
                            const float2 y = unpack2(x), e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                            if (j & 1) sum1 = add2(sum1, pack2(e.x, e.y)); else sum0 = add2(sum0, pack2(e.x, e.y));
                            w16[j] = Half2<T>::narrow(e.x, e.y);
                        }
                        tmem_st16(s_at + (i / 2) * 64 + (i & 1) * 16, w16);
                        if (kParts == 2 && i == 1) {  // the first 64 keys' weights can go
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars.p_full[m_tile][0]);
                        }
                    }
                    sum = add2(sum, add2(sum0, sum1));
                    tmem_wait_st();
                } else if (S::kPaired) {
                    // A pair without rows here meets too, as one with rows does
                    // at its first tile: the first half's hand-over alone lets
                    // the product write all channels, and the other half may
                    // still be reading those of the block before.
                    if (t == w.t0) pair_sync(pair);
                } else if (lane == 0) {
                    mbar_arrive(&bars.p_full[m_tile][0]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[m_tile][kParts == 2 ? 1 : half]);
            }
            wait_or_fail(&bars.pv_done[m_tile], (n - 1) & 1, watch, limit);
            tc_fence_after();
            if (!warp_live) continue;
            const float2 both = unpack2(sum);
            float l = both.x + both.y;
            if constexpr (S::kPaired) {
                *swap_mine = l;
                pair_sync(pair);
                l = half ? *swap_other + l : l + *swap_other;
                pair_sync(pair);  // read by both before it is written again
            }
            const bool mine = row < rows;
            const uint32_t token = (uint32_t)w.q.q0 + first + my_token, head = w.head * p.group + my_head;
            const float ref = reference<T>(m, p.c);  // log2 units
            const bool whole = w.starts && w.ends, any = begin < stop;
            const float inv = any ? 1.0f / l : 0.0f;
            uint16_t *const out = (uint16_t *)p.a.d_out + (uint64_t)token * p.a.out_stride[0] + (uint64_t)head * p.a.out_stride[1];
            float *const part = p.parts + (size_t)(blockIdx.x * 2 + (w.starts ? 1 : 0)) * S::kPartFloats;
            // a NaN that the sum does not have: from a hidden key's values?
            uint64_t seen = pack2(0.0f, 0.0f);
#pragma unroll 1
            for (uint32_t i = 0; i < kOwn / 32; ++i) {
                uint32_t o[32];
                tmem_ld32(o_at + i * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) seen = add2(seen, pack2(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1])));
            }
            const float2 seen2 = unpack2(seen);
            const bool odd = mine && seen2.x + seen2.y != seen2.x + seen2.y && l == l && failed == 0;
            // where the output lies over the queries, neither of a pair may
            // write before both have read
            const bool wait_both = S::kPaired && whole && (const void *)p.a.d_out == p.a.d_q && pair_any(pair, odd);
            if (__any_sync(0xFFFFFFFFu, odd))
                mend_rows<T, D, (int)kOwn>(&p, &control.watch, w.r, w.head, (const uint16_t *)p.a.d_q + (uint64_t)token * p.a.q_stride[0] + (uint64_t)head * p.a.q_stride[1],
                                           odd, max(begin, w.t0 * (int32_t)p.key_tile), min(stop, w.t1 * (int32_t)p.key_tile), m == -INFINITY ? 0.0f : ref, o_at, half * kOwn);
            if (wait_both) pair_sync(pair);
            if (whole) {
#pragma unroll
                for (int i = 0; i < (int)kOwn / 32; ++i) {
                    uint32_t o[32];
                    tmem_ld32(o_at + i * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = any ? __uint_as_float(o[8 * j + e]) * inv : 0.0f;
                        if (mine) *(uint4 *)(out + half * kOwn + i * 32 + j * 8) = narrow8<T>(x);
                    }
                }
                if (half == 0 && row < rows && p.a.d_lse_or_null)
                    p.a.d_lse_or_null[(uint64_t)token * p.a.q_heads + head] = any ? (l > 0.0f || l != l ? (ref + log2f(l)) * kLn2 : -INFINITY) : -INFINITY;
            } else {
#pragma unroll
                for (int i = 0; i < (int)kOwn / 32; ++i) {
                    uint32_t o[32];
                    tmem_ld32(o_at + i * 32, o);
                    tmem_wait_ld();
                    if (mine)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *(uint4 *)(part + S::part_o(m_tile, half * (kOwn / 4) + i * 8 + j, row)) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
                if (half == 0 && row < rows) *(float2 *)(part + S::part_ml(m_tile, row)) = make_float2(m == -INFINITY ? -INFINITY : ref, l);
            }
            tc_fence_before();
        }
        tc_fence_before();
    }
    if (wid == S::kStatusWarp) {  // the requests' statuses, a request per CTA at a time
        for (uint32_t r = blockIdx.x; r < p.kv.n_reqs; r += gridDim.x) {
            const Request q = load_request(p.kv, r);
            sz_status st = q.status;
            if (st == SZ_OK && q.n > 0 && q.kv > 0) {
                int32_t begin, stop;
                key_range(p, q, 0, q.n, &begin, &stop);
                st = check_pages(p.kv, r, (uint32_t)begin / p.kv.page_tokens, (uint32_t)(q.kv - 1) / p.kv.page_tokens + 1);
            }
            if (lane == 0) {
                p.status[r] = st;
                __threadfence();  // a CTA that fails sets timed_out, then the statuses
                if (timed_out(p)) p.status[r] = SZ_ERR_DEVICE_TIMEOUT;
            }
        }
    }
    // ------------------------------------------------------------------ end
    __syncthreads();
    if (failed) {  // rows may be unfinished: no result of this call stands
        // Products and copies under way must end before the memory that they
        // write is given back.  They get a second, however short the limit.
        const uint64_t patience = umax64(limit, kLandingNs);
        if (wid >= kMmaWarp && wid < kMmaWarp + S::kMmaWarps) {
            uint64_t *const drain = &bars.drain[wid - kMmaWarp];
            if (elect_one()) {
                mma_commit(drain);
                mbar_wait(drain, 0, patience);
            }
            __syncwarp();
        }
        if (wid == S::kKeyWarp) {
            const uint32_t kinds = (p.debug_flags & kDebugNoSignal) != 0 ? 1 : 2;
            for (uint32_t kind = 0; kind < kinds; ++kind) {  // the last use of each slot is among these
                const uint32_t end = control.issued[kind];
                for (uint32_t u = end > 2 * S::kSlots ? end - 2 * S::kSlots : kind; u < end; u += 2)
                    mbar_wait(&bars.full[u % S::kSlots], u / S::kSlots & 1, patience);
            }
            const uint32_t end = control.queries;
            for (uint32_t u = end > S::kQueries ? end - S::kQueries : 0; u < end; ++u)
                mbar_wait(&bars.q_full[u % S::kQueries], u / S::kQueries & 1, patience);
        }
        if (tid == 0) {
            *(volatile unsigned long long *)(p.timed_out + 1) = globaltimer_ns();
            __threadfence();
            atomicExch(p.timed_out, p.call);
            __threadfence();
        }
        __syncthreads();
        for (uint32_t r = tid; r < p.kv.n_reqs; r += S::kThreads) p.status[r] = SZ_ERR_DEVICE_TIMEOUT;
    }
    if (wid == kMmaWarp) tmem_free(tmem, S::kColumns);
}

// Join the parts of split blocks.  Two parts join like two sets of keys:
// (m, l, o) and (m', l', o') to M = max, l 2^(m - M) + l' 2^(m' - M), the
// same for o.  What bounds it is the latency of its few loads, so it is spread
// out: a block of threads per CTA that began a split block, row tile and
// D/8 channels; a thread holds one row's and, where rows are few (a decode
// step, whose parts are many), one slice of the parts.  Slices and parts are
// added in a fixed order.  It takes 4 to 8 us behind the kernel above, its
// launch overlapped; joining in the last CTA to arrive, behind a counter and
// fences, took longer.
constexpr int kJoinThreads = 128;
constexpr uint32_t kJoinGroups = 8;

template <typename T, int D, int kM>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const __grid_constant__ TensorArgs p) {
    using S = Shape<D, kM>;
    constexpr int kChunks = D / 4 / (int)kJoinGroups, kBatch = 4;
    __shared__ float shared[kJoinThreads][kChunks * 4 + 3];
    const uint32_t tid = threadIdx.x, c0 = blockIdx.x, chunk = blockIdx.y * kChunks, m_tile = blockIdx.z;
    grid_dependency_wait();
    if (c0 == 0 && blockIdx.y == 0 && m_tile == 0 && tid == 0) *p.timed_out = 0;  // every CTA has looked
    const SplitRec w = p.rec[c0];
    if (w.last <= c0 || w.last >= p.ctas) return;
    const uint32_t first = (w.block * kM + m_tile) * p.tile_tokens;
    if ((uint32_t)w.q.n <= first) return;
    const uint32_t rows = umin32((uint32_t)w.q.n - first, p.tile_tokens) * p.group, parts = w.last - c0 + 1;
    const uint32_t row_span = rows <= 1 ? 1u : 1u << (32 - __clz(rows - 1)), slices = kJoinThreads / row_span;
    const uint32_t row = tid % row_span, slice = tid / row_span;
    const float *const base = p.parts + (size_t)(c0 * 2) * S::kPartFloats;  // part 0 is the first CTA's second slot
    float top = -INFINITY, sum = 0.0f, o[kChunks][4] = {};
    for (uint32_t k0 = slice; k0 < parts && row < rows; k0 += kBatch * slices) {
        float4 v[kBatch][kChunks];
        float2 ml[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t k = umin32(k0 + i * slices, parts - 1);
            const float *from = base + (size_t)(k == 0 ? 1 : 2 * k) * S::kPartFloats;
            ml[i] = __ldcg((const float2 *)(from + S::part_ml(m_tile, row)));
            if (k0 + i * slices >= parts) ml[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int j = 0; j < kChunks; ++j) v[i][j] = __ldcg((const float4 *)(from + S::part_o(m_tile, chunk + j, row)));
        }
        float high = top;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) high = fmaxf(high, ml[i].x);
        const float keep = high == top ? 1.0f : exp2f(top - high);
        top = high;
        sum *= keep;
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] *= keep;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (k0 + i * slices >= parts) continue;
            // where nothing is visible, or all of it scored -inf, the part holds
            // zeros, or NaN of a value that is not finite
            const float f = ml[i].x == -INFINITY ? 0.0f : exp2f(ml[i].x - top);
            sum += ml[i].y * f;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                o[j][0] += v[i][j].x * f;
                o[j][1] += v[i][j].y * f;
                o[j][2] += v[i][j].z * f;
                o[j][3] += v[i][j].w * f;
            }
        }
    }
    if (slices > 1) {
        float *const mine = shared[tid];
#pragma unroll
        for (int j = 0; j < kChunks * 4; ++j) mine[j] = o[j / 4][j % 4];
        mine[kChunks * 4] = top;
        mine[kChunks * 4 + 1] = sum;
        __syncthreads();
        if (slice == 0)
            for (uint32_t k = 1; k < slices && k < parts; ++k) {
                const float *const from = shared[k * row_span + row];
                const float high = fmaxf(top, from[kChunks * 4]);
                const float keep = high == top ? 1.0f : exp2f(top - high), f = from[kChunks * 4] == -INFINITY ? 0.0f : exp2f(from[kChunks * 4] - high);
                top = high;
                sum = sum * keep + from[kChunks * 4 + 1] * f;
#pragma unroll
                for (int j = 0; j < kChunks * 4; ++j) o[j / 4][j % 4] = o[j / 4][j % 4] * keep + from[j] * f;
            }
    }
    if (slice != 0 || row >= rows) return;
    const uint32_t tok = row / p.group;
    int32_t begin, stop;
    key_range(p, w.q, (int32_t)(first + tok), (int32_t)(first + tok) + 1, &begin, &stop);
    const bool any = begin < stop;
    const float inv = any ? 1.0f / sum : 0.0f;
    const uint32_t token = (uint32_t)w.q.q0 + first + tok, head = w.head * p.group + row % p.group;
    uint16_t *out = (uint16_t *)p.a.d_out + (uint64_t)token * p.a.out_stride[0] + (uint64_t)head * p.a.out_stride[1] + chunk * 4;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        uint2 x = make_uint2(0u, 0u);
        if (any) x = make_uint2(Half2<T>::narrow(o[j][0] * inv, o[j][1] * inv), Half2<T>::narrow(o[j][2] * inv, o[j][3] * inv));
        ((uint2 *)out)[j] = x;
    }
    if (chunk == 0 && p.a.d_lse_or_null)
        p.a.d_lse_or_null[(uint64_t)token * p.a.q_heads + head] = any && sum != 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------- host side
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            fn = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(fn);
    }();
    return f;
}

// A map over `rank` dimensions, channels first.  A dimension of size 1 may
// come with any stride; the map gets a legal one.
static bool make_map(CUtensorMap *map, uint32_t dtype, void *base, int rank, const uint64_t *size, const uint64_t *stride_elems,
                     const uint32_t *box) {
    cuuint64_t dims[4], strides[3];
    cuuint32_t boxes[4], steps[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        dims[i] = size[i];
        boxes[i] = box[i];
        if (i) strides[i - 1] = size[i] > 1 ? stride_elems[i] * 2 : size[0] * 2;
    }
    return encode_tiled()(map, dtype == SZ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
                          base, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Let `Kernel` use `bytes` of dynamic shared memory, asked once per device.
template <auto Kernel>
static cudaError_t allow_shared(uint32_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (const cudaError_t e = cudaGetDevice(&dev)) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Which shapes the tensor-core kernel takes: heads of 64 or 128 channels, a
// positive scale (the running maximum is of unscaled scores) whose products
// with a score or with the difference of two neither vanish nor lose bits
// before these overflow, row tiles that hold a whole group, and pages whose
// copies start on a swizzle group of 8 rows and fill or divide a tile.
static bool tensor_shape(const sz_paged_kv &kv, const sz_attention_args &a) {
    if (kv.head_dim != 64 && kv.head_dim != 128) return false;
    if (!(a.scale >= 1e-30f) || !(a.scale < 1e30f)) return false;
    if (a.q_heads / kv.heads > kTileRows || kv.n_pages == 0 || kv.n_tokens == 0) return false;
    // queries repeated over heads or tokens, or lying over one another: a
    // tensor map's rows do not overlap
    if ((a.q_heads > 1 && a.q_stride[1] < kv.head_dim) || (kv.n_tokens > 1 && a.q_stride[0] < kv.head_dim)) return false;
    return kv.page_tokens % 8 == 0 && (kv.page_tokens <= kTileRows || kv.page_tokens % kTileRows == 0);
}

template <int D, int kM>
static uint64_t tensor_workspace() {
    const uint64_t ctas = (uint64_t)kMaxTensorSms * Shape<D, kM>::kCtasPerSm;
    return 16 + ctas * sizeof(SplitRec) + 2 * 4ull * Shape<D, kM>::kPartFloats * ctas;
}

// A tag for a call's words in the workspace: 48 bits, from a start of the
// clocks and the process (nothing that can throw), so
// that words of earlier calls, or of other memory, do not carry it.
static unsigned long long next_call() {
    static std::atomic<unsigned long long> next{[] {
        unsigned long long x = (unsigned long long)std::chrono::system_clock::now().time_since_epoch().count() ^
                               (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() << 20 ^
                               (unsigned long long)getpid() << 44;
        x = (x ^ x >> 31) * 0x9E3779B97F4A7C15ull;  // every bit of the clocks reaches the 48 kept
        return x ^ x >> 29;
    }()};
    for (;;)
        if (const unsigned long long tag = next.fetch_add(1) & 0xFFFFFFFFFFFFull) return tag;
}

uint64_t attention_workspace(uint32_t head_dim) {
    if (head_dim == 128) return umax64(tensor_workspace<128, 1>(), tensor_workspace<128, 2>());
    if (head_dim == 64) return umax64(tensor_workspace<64, 1>(), tensor_workspace<64, 2>());
    return 256;
}

template <typename T, int D, int kM>
static cudaError_t launch_tensor(const sz_paged_kv &kv, const sz_attention_args &a, int32_t *status, void *ws, const DeviceInfo &dev,
                                 cudaStream_t s) {
    using S = Shape<D, kM>;
    TensorArgs p{};
    p.kv = kv;
    p.a = a;
    p.c = a.scale * kLog2e;
    p.group = a.q_heads / kv.heads;
    p.tile_tokens = S::kRows / p.group;
    p.box_tokens = umin32(kv.page_tokens, kTileRows);
    p.copies = kTileRows / p.box_tokens;
    p.key_tile = p.copies * p.box_tokens;
    p.ctas = umin32((uint32_t)dev.sms, kMaxTensorSms) * S::kCtasPerSm;
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.parts = reinterpret_cast<float *>(at);
    at += (size_t)p.ctas * 2 * 4 * S::kPartFloats;
    p.timed_out = reinterpret_cast<unsigned long long *>(at);
    // Where the sizes known here already say that no block will be split
    // (find_share comes to the same), nothing needs joining.
    const uint64_t span = (uint64_t)S::kTiles * p.tile_tokens, blocks = kv.heads * (kv.n_reqs + kv.n_tokens / span);
    const bool split = blocks > p.ctas || div_up((uint64_t)kv.max_pages * kv.page_tokens, p.key_tile) > kWholeTiles;
    const uint64_t most = div_up((uint64_t)kv.max_pages * kv.page_tokens, p.key_tile) + 1 + kBlockUnits<D, kM>;  // units of a block
    const bool wide = blocks >= (1ull << 32) / (p.ctas + 1) / most;  // units times CTAs may pass 32 bits
    p.rec = split ? reinterpret_cast<SplitRec *>(at + 16) : nullptr;
    p.call = next_call();
    p.status = status;
    p.wait_limit_ns = wait_limit_ns();
    p.debug_flags = debug_flags();
    CUtensorMap q_map, k_map, v_map;
    const uint64_t q_size[3] = {D, a.q_heads, kv.n_tokens}, q_stride[3] = {1, a.q_stride[1], a.q_stride[0]};
    const uint32_t q_box[3] = {64, p.group, p.tile_tokens};
    const uint64_t size[4] = {D, kv.page_tokens, kv.heads, kv.n_pages};
    const uint64_t k_stride[4] = {1, kv.k_stride[2], kv.k_stride[1], kv.k_stride[0]};
    const uint64_t v_stride[4] = {1, kv.v_stride[2], kv.v_stride[1], kv.v_stride[0]};
    const uint32_t box[4] = {64, p.box_tokens, 1, 1};
    if (!encode_tiled() || !make_map(&q_map, kv.dtype, const_cast<void *>(a.d_q), 3, q_size, q_stride, q_box) ||
        !make_map(&k_map, kv.dtype, kv.d_k, 4, size, k_stride, box) || !make_map(&v_map, kv.dtype, kv.d_v, 4, size, v_stride, box))
        return cudaErrorInvalidValue;
    if (wide) {
        if (const cudaError_t e = allow_shared<attention_kernel<T, D, kM, uint64_t>>(S::kSmem)) return e;
        attention_kernel<T, D, kM, uint64_t><<<p.ctas, S::kThreads, S::kSmem, s>>>(p, q_map, k_map, v_map);
    } else {
        if (const cudaError_t e = allow_shared<attention_kernel<T, D, kM, uint32_t>>(S::kSmem)) return e;
        attention_kernel<T, D, kM, uint32_t><<<p.ctas, S::kThreads, S::kSmem, s>>>(p, q_map, k_map, v_map);
    }
    if (const cudaError_t e = cudaGetLastError()) return e;
    if (!split) return cudaSuccess;
    return launch_after(attention_join_kernel<T, D, kM>, dim3(p.ctas, kJoinGroups, kM), dim3(kJoinThreads), 0, s, p);
}

template <typename T>
static cudaError_t launch_attention_t(const sz_paged_kv &kv, const sz_attention_args &a, int32_t *status, void *ws, const DeviceInfo &dev,
                                      cudaStream_t s) {
    if (!tensor_shape(kv, a)) return launch_any_t<T>(kv, a, status, s);
    // Two row tiles per CTA share a key tile; with no more rows per request
    // than one short tile holds (on average: the lengths are on the device),
    // two CTAs per SM of one row tile each keep more copies in flight.  Both
    // ways, one and two row tiles: 64 requests of one token 129 and 149 us,
    // one token over 131,071 keys 93 and 105, 16 requests of 5 tokens and 8
    // heads 45 and 50; a 4,096 x 32,768 chunk 3.56 and 1.66 ms, ragged
    // prompts 127 and 63 us, a 2,048-token chunk behind a window 504 and 266.
    const uint64_t group = a.q_heads / kv.heads, rows = kv.n_tokens * group;
    const bool two = rows > (uint64_t)kv.n_reqs * 64 || group > 64;
    if (kv.head_dim == 128)
        return two ? launch_tensor<T, 128, 2>(kv, a, status, ws, dev, s) : launch_tensor<T, 128, 1>(kv, a, status, ws, dev, s);
    return two ? launch_tensor<T, 64, 2>(kv, a, status, ws, dev, s) : launch_tensor<T, 64, 1>(kv, a, status, ws, dev, s);
}

cudaError_t launch_attention(const sz_paged_kv &kv, const sz_attention_args &a, int32_t *status, void *ws, const DeviceInfo &dev,
                             cudaStream_t s) {
    return kv.dtype == SZ_BF16 ? launch_attention_t<__nv_bfloat16>(kv, a, status, ws, dev, s)
                               : launch_attention_t<__half>(kv, a, status, ws, dev, s);
}

}  // namespace sz
