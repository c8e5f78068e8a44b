// kvo_paged_chunk_attn: attention of several new tokens of each request over a paged cache (bf16, or e4m3 with a scale per
// page and KV head) that holds them already.
//
//   o_i = sum_t softmax_t(q_i . k_t / sqrt(d)) v_t,  t <= len - n + i  for the i-th of n new tokens of len.
//
// Work.  An item is a block of 256 query rows of one KV head: two tiles of 128 rows, each floor(128 / r) tokens x the r
// query heads of the group (one tile where the tokens fit it), over the keys that they see, 128 to a tile.  The items of
// all requests, laid end to end by an estimate of their cost, are cut into equal ranges, one per CTA and SM; the lengths
// are device data, so each CTA finds its range by a prefix sum over the requests.  An item that a border cuts leaves its
// parts (m, l, o in fp32) in the workspace and a second kernel joins them in the order of the keys: results do not depend
// on timing.
//
// One CTA to an SM, its warps
//   9        walks the items: their descriptors, tiles of K, and of e4m3 V, through rings (TMA, a box per page), the pages' scales,
//   11       (bf16) tiles of V,
//   8, 10    one thread each issues the tcgen05.mma of tile 0 and 1: S_t = Q_t K^T and O_t += P_t V,
//   0-3, 4-7 the softmax of tile 0 and 1, one thread per row: S from tensor memory, online maximum and sum in fp32, P (bf16, or
//            f16 next to e4m3) back over S,
//   12-15    (e4m3) V to f16.
// An item's first scores are issued behind the last value product of the one before, and its first loads before that.
//
// e4m3.  K goes to the tensor cores as it is: a row of q, times a power of two that brings its largest value to 2^7..2^8, is
// the sum of two e4m3 values, exactly for what is at least 2^-9 of that largest and to 2^-17 of it for all below (a bf16
// value has 8 bits, an e4m3 value 4), and two 8-bit products take the time of one of bf16.  V is widened to f16, exactly, on its
// way through shared memory.  A page's k_scale multiplies its scores; its v_scale goes into the exponents of its weights,
// exp2(s + log2 v_scale - m) with m the maximum of those, so that f16 holds what contributes most whatever the scales are.
// The sum l of the exponentials without v_scale takes each page's share times 2^c / v_scale, in fp32: l counts in units of
// 2^(m - c), with 2^c about the first page's scale, or what keeps l in fp32's range where scales differ by more than 2^32; c
// is a whole number, so that o = (sum of weights and codes) / l * 2^c takes no further rounding.
//
// What bounds it.  Long chunks: the tensor cores, which wait for the softmax (two tiles in turn, a row to a thread) at the
// hand-overs.  32 query heads over 8 of d 128: 8192 tokens alone in bf16 390 us, 1.41 PFLOP/s of 1.91 measured for a matrix
// product, in e4m3 478; 2048 behind 30000 in bf16 665 us (1.57 PFLOP/s), in e4m3 820: there the conversions of V and of P and
// more code than the instruction caches hold.  Few rows on many keys: the loads of K and V, 16 requests of 64 tokens behind 32k
// in bf16 385 us, 5.6 TB/s.  A batch of both, 36 single tokens and 4 chunks: 161 us replayed, 170 called, 0.90 PFLOP/s.  Of d 64
// the products take half and the softmax what it takes: 8192 tokens 343 us in bf16, 417 in e4m3.
//
// Why so.  One thread for both tiles' products kept one tile waiting for the other's barriers: 8192 tokens 440 -> 402 us with
// two.  Two buffers of f16 V: 2048 e4m3 tokens behind 30000 965 us, three 787.  q split into its pieces by every CTA that
// needs them: 8192 tokens 744 us, by a launch before 457.  The softmax unrolled over 128 keys: 1016 us, in loops 740.  One
// warp that loads both K and V keeps K waiting behind V's buffers: in bf16 the mixed batch 251 us, with two 166; in e4m3 the
// buffers of raw V are free early, and a second warp's code costs more: 2048 behind 30000 945 us, with one 810.  K asked for
// before its tile's scales are read: 16 pieces of 8 tokens behind 32k in e4m3 265 -> 250 us.
#include <algorithm>

#include "f32x2.cuh"
#include "kvo_internal.cuh"
#include "launch.cuh"
#include "paged.cuh"
#include "paged_few.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace kvo {

size_t round256(size_t x);

constexpr int CH_ROWS = 128;               // query rows of a tile
constexpr int CH_KEYS = 128;               // keys of a tile
constexpr int CH_BLOCK = CH_ROWS * 128;    // bytes of 128 rows of 128
constexpr float CH_RAISE = 8.f;            // log2: how far a score may pass the running maximum
template <bool FP8>
constexpr float CH_BIAS_OF = FP8 ? 6.f : 0.f;          // log2: weights are held times 2^this; in f16, whose smallest step is 2^-24
constexpr float CH_BIG = 0x1p20f;          // from here on scores are taken less the maximum before anything is added to them
constexpr int CH_CTAS = 152;               // ranges at most: one CTA to an SM
constexpr int CH_EVENTS = 16;              // barriers that a tile's products complete in turn
constexpr int CH_ITEMS = 4;                // descriptors
constexpr int CH_NAN = -128;               // the exponent of a row of q that is not finite
constexpr int CH_SCALES = 8;               // tiles of keys whose scales are held
constexpr uint32_t CH_FAR = 1u << 8;       // beside a tile's bad groups: some v_scale of the item so far is far from its first,
constexpr float CH_SPREAD = 32.f;          // log2: that is, further than this
constexpr float CH_NEAR = 40.f;            // log2: where l takes 2^-c at an item's end
constexpr float CH_NO_SCALE = -160.f;      // log2 of a v_scale of 0: 2^-160 times any code is 0 in fp32
constexpr float CH_TOP_C = 256.f;          // above any c that a page asks for

template <int D, bool FP8>
struct ChShape;
template <int D>
struct ChShape<D, false> {
    static constexpr int THREADS = 384;
    static constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 88;
    static constexpr int Q = CH_ROWS * D * 2;                   // bytes of a tile of q
    static constexpr int TILE = CH_KEYS * D * 2;                // of K or V
    static constexpr int KS = D == 128 ? 2 : 4, VS = KS;        // stages of K and of V: even numbers (see `dual`)
    static constexpr int WIDE_BYTES = 0, WIDES = 1;
    static constexpr int TILES = 2 * Q + (KS + VS) * TILE;
};
template <int D>
struct ChShape<D, true> {
    static constexpr int THREADS = 512;
    static constexpr int REGS_SOFTMAX = 168, REGS_OTHER = 88;
    static constexpr int Q = 2 * CH_ROWS * D;                   // the two pieces
    static constexpr int TILE = CH_KEYS * D;                    // of K or V as they are
    static constexpr int WIDE_BYTES = CH_KEYS * D * 2;          // of V in f16
    static constexpr int KS = D == 128 ? 2 : 4, VS = 2;
    static constexpr int WIDES = 3;                             // (any number: tiles are widened in their order)
    static constexpr int TILES = 2 * Q + (KS + VS) * TILE + WIDES * WIDE_BYTES;
};

struct ChunkArgs {
    const int8_t* q_exp;           // e4m3 pages: q's pieces are its values times 2^this
    const float* k_scale;
    const float* v_scale;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;
    uint16_t* o;
    float* lse;                    // or NULL
    int32_t* status;
    struct ChunkCut* cut;          // [CTAs]
    float* part_o;                 // [CTAs][2][tiles][D / 4][128] of 4 values
    void* part_ml;                 // [CTAs][2][tiles][128]: m, l (float2) or, next to e4m3 pages, m, l, c (float4)
    int64_t total;
    int batch, hq, hkv, r, tq, page, shift, n_pages, max_pages, tiles;
    int w1, w2, base;              // cost of a key for one tile of rows and for two, and of an item in itself
    int64_t least;                 // cost of a range, unless there are more than CTAs
    float scale_log2;
    int wide;                      // o is 32-byte aligned
    int skip;                      // the load that every CTA announces without copying it (tests; -1: none)
    long long wait_ns;
};

// What a CTA tells the join: the item that begins in its range and ends in a later one.
struct ChunkCut {
    int64_t row;                   // the request's first row of q
    int32_t last;                  // the range in which it ends; -1: no such item
    int32_t more;                  // whether this CTA's range begins with a part of an item that began before
    int32_t tok0, n, g;            // first token of the block, the request's tokens, KV head
};

struct ChunkItem {
    int64_t row;
    int32_t n0, n1;                // tiles of keys of each tile of rows; n0 = -1: the end
    int32_t tiles;                 // of keys in all
    int32_t dual;                  // one tile of rows only: both take it, with the even and the odd tiles of keys
    int32_t first;                 // tile of keys
    int32_t b, g, tok0, nq, len;
    int32_t part;                  // -1: the whole item; else its place in the workspace
    // The completions of a tile of rows' products are counted: its scores with the i-th of its tiles of keys (value 0) and
    // the value product after them (1).  One commit for the next scores stands for a value product as well, where the
    // other tile's products run meanwhile; a dual item's stages of V would wait for it too long.
    __device__ __forceinline__ uint32_t event(int i, int value) const { return dual ? 2 * i + value : i + value; }
    __device__ __forceinline__ int n(int t) const { return t ? n1 : n0; }       // (an array would live in local memory)
    __device__ __forceinline__ uint32_t events(int t) const { return n(t) == 0 ? 0 : event(n(t) - 1, 1) + 1; }
};

struct ChShared {
    uint64_t q_full[2], k_full[4], v_full[4], raw_free[2], wide_full[3], event[2][CH_EVENTS], p_full[2][2], turn[2], drain[2], v_tail, item_full[CH_ITEMS],
        item_free[CH_ITEMS], sc_full[CH_SCALES], ml_there, weights_there, o_read;
    ChunkItem item[CH_ITEMS];
    alignas(16) float k_scale[CH_SCALES][8];
    alignas(16) float v_log[CH_SCALES][8];          // of each 16 keys of a tile: k_scale, log2 of v_scale
    alignas(16) float v_share[CH_SCALES][8];        // 2^v_first over v_scale; 0 from CH_FAR on
    uint2 bad[CH_SCALES];          // groups of 16 keys in pages that do not exist, and CH_FAR; log2 of the item's first v_scale, rounded
    uint32_t tmem;
    int abort;
    int k_issued, v_issued, tail_open, tail_phase, q_issued[2];
    union {
        struct {                   // the plan
            int64_t sum[16], at[2];
            int32_t top[16], found[2], high[2];
        };
        struct {                   // the two halves of a dual item: maximum, sum and c one way, weights and c the other
            float2 share[CH_ROWS];
            int16_t share_c[CH_ROWS];
        };
    };
};

// Whole warp: true for one of its threads, the same each time; the compiler knows that it is one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ bool ch_wait_long(int* abort, int32_t* status, uint32_t bar, uint32_t parity, long long limit) {
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*(volatile int*)abort) return false;
        if ((long long)(global_ns() - t0) > limit) {
            *(volatile int*)abort = 1;
            if (status) atomicOr(status, KVO_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool ch_wait(ChShared& sh, const ChunkArgs& A, uint64_t& bar, uint32_t parity) {
    const uint32_t b = smem_u32(&bar);
    if (mbar_try_wait(b, parity & 1)) return true;
    return ch_wait_long(&sh.abort, A.status, b, parity & 1, A.wait_ns);
}
// The e-th completion of tile t's products: its scores of each tile of keys, then its last value product, item after item.
__device__ __forceinline__ bool ch_event(ChShared& sh, const ChunkArgs& A, int t, uint32_t e) {
    return ch_wait(sh, A, sh.event[t][e % CH_EVENTS], e / CH_EVENTS);
}

// ------------------------------------------------------------------ the plan
struct ChRequest {
    int a, n, len;                 // first row, new tokens, tokens in all
    bool served;
};
// Cost of the first i blocks of a request, all but its last, and of one of them; for all KV heads.
__device__ __forceinline__ int64_t ch_before(const ChunkArgs& A, const ChRequest& r, int64_t i) {
    const int64_t past = max(r.len - r.n, 0);
    return A.hkv * (i * (A.base + A.w2 * past) + (int64_t)A.w2 * A.tq * i * (i + 1));
}
__device__ __forceinline__ int ch_blocks(const ChunkArgs& A, const ChRequest& r) { return (r.n + 2 * A.tq - 1) / (2 * A.tq); }
// Cost of one item of block i.
__device__ __forceinline__ int64_t ch_cost(const ChunkArgs& A, const ChRequest& r, int i) {
    const int64_t past = max(r.len - r.n, 0), end = min((int64_t)(i + 1) * 2 * A.tq, (int64_t)r.n);
    return A.base + (end - (int64_t)i * 2 * A.tq > A.tq ? A.w2 : A.w1) * (past + end);
}
__device__ __forceinline__ int64_t ch_total(const ChunkArgs& A, const ChRequest& r) {
    if (!r.served || r.n == 0) return 0;
    const int nb = ch_blocks(A, r);
    return ch_before(A, r, nb - 1) + A.hkv * ch_cost(A, r, nb - 1);
}
// Tiles of keys that tile t of rows of block i sees.
__device__ __forceinline__ int ch_tiles(const ChunkArgs& A, const ChRequest& r, int i, int t) {
    const int first = (i * 2 + t) * A.tq, have = min(r.n - first, A.tq);
    if (have <= 0) return 0;
    const int64_t see = (int64_t)first + have + r.len - r.n;
    return (int)((max(see, (int64_t)0) + CH_KEYS - 1) / CH_KEYS);
}

struct ChWalk {                    // a place in the list of items
    ChRequest r;
    int b, i, g;
    int64_t start, cost;           // of the item
};
// The item of request b (which begins at `at`) that holds position x.
__device__ __forceinline__ ChWalk ch_locate(const ChunkArgs& A, int b, const ChRequest& r, int64_t at, int64_t x) {
    int lo = 0, n = ch_blocks(A, r);
    while (n > 1) {
        const int half = n / 2;
        if (at + ch_before(A, r, lo + half) <= x) { lo += half; n -= half; }
        else n = half;
    }
    ChWalk w;
    w.r = r;
    w.b = b;
    w.i = lo;
    w.cost = ch_cost(A, r, lo);
    at += ch_before(A, r, lo);
    w.g = (int)((x - at) / w.cost);
    w.start = at + w.g * w.cost;
    return w;
}
// Which of an item's n tiles of keys lie in [lo, hi).
__device__ __forceinline__ void ch_part(const ChWalk& w, int64_t lo, int64_t hi, int n, int& first, int& last) {
    first = w.start >= lo ? 0 : (int)((lo - w.start) * n / w.cost);
    last = w.start + w.cost <= hi ? n : (int)((hi - w.start) * n / w.cost);
}
__device__ __forceinline__ ChRequest ch_request(const ChunkArgs& A, int b) {
    const int a = A.cu[b], e = A.cu[b + 1], len = A.lens[b];
    return {a, e - a, (int)min((int64_t)max(len, 0), (int64_t)A.max_pages * A.page), offsets_ascend(a, e, A.total)};
}
__device__ __forceinline__ int64_t ch_bound(int64_t total, int ranges, int c) { return total / ranges * c + total % ranges * c / ranges; }

struct ChPlan {
    int64_t all;                   // the cost of everything
    int64_t lo, hi;                // this CTA's range
    int ranges;
};
// All threads.  Finds this CTA's range and the requests that hold its first and last position; false where it has none.
template <int THREADS>
__device__ __forceinline__ bool ch_plan(ChShared& sh, const ChunkArgs& A, ChPlan& plan) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int WARPS = THREADS / 32;
    int64_t total = 0;
    int top = 0;                   // the end of the served requests so far
    ChRequest mine;
    int64_t before = 0, cost = 0;
    int top_before = 0;
    // Adds the next THREADS requests: this thread's cost and what lies before it.
    auto add = [&](int base, bool report) {
        const int b = base + tid;
        mine = {0, 0, 0, false};
        if (b < A.batch) {
            mine = ch_request(A, b);
            const int len = A.lens[b];
            if (report && A.status && (!mine.served || len < 0 || len > (int64_t)A.max_pages * A.page)) atomicOr(A.status, KVO_DEV_BAD_COUNT);
        }
        int m = mine.served ? mine.a + mine.n : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o) m = max(m, x);
        }
        int m_before = __shfl_up_sync(0xffffffffu, m, 1);
        if (lane == 0) m_before = 0;
        __syncthreads();
        if (lane == 31) sh.top[warp] = m;
        __syncthreads();
        top_before = top;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) top_before = max(top_before, sh.top[w]);
            top = max(top, sh.top[w]);
        }
        top_before = max(top_before, m_before);
        mine.served = mine.served && mine.a >= top_before;
        cost = ch_total(A, mine);
        int64_t s = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        if (lane == 31) sh.sum[warp] = s;
        __syncthreads();
        before = total + s - cost;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += sh.sum[w];
            total += sh.sum[w];
        }
    };
    for (int base = 0; base < A.batch; base += THREADS) add(base, blockIdx.x == 0);
    plan.all = total;
    plan.ranges = (int)min((int64_t)gridDim.x, max(total / A.least, (int64_t)1));
    const int c = blockIdx.x;
    if (c >= plan.ranges || total == 0) return false;
    const int64_t border = ch_bound(total, plan.ranges, c + (lane & 1));
    plan.lo = __shfl_sync(0xffffffffu, border, 0);
    plan.hi = __shfl_sync(0xffffffffu, border, 1);
    if (plan.lo >= plan.hi) return false;
    auto look = [&](int base) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t x = k ? plan.hi - 1 : plan.lo;
            if (before <= x && x < before + cost) {
                sh.found[k] = base + tid;
                sh.at[k] = before;
                sh.high[k] = top_before;
            }
        }
    };
    if (A.batch <= THREADS) {
        look(0);
    } else {
        total = 0;
        top = 0;
        for (int base = 0; base < A.batch; base += THREADS) {
            add(base, false);
            look(base);
        }
    }
    return true;                   // (what was found is there after a barrier)
}
// What the join has to know of this CTA's range, which begins with item `head`.
__device__ __forceinline__ ChunkCut ch_cut(const ChShared& sh, const ChunkArgs& A, const ChPlan& P, const ChWalk& head) {
    ChunkCut cut;
    const ChWalk tail = ch_locate(A, sh.found[1], ch_request(A, sh.found[1]), sh.at[1], P.hi - 1);
    int first, last, n = max(ch_tiles(A, head.r, head.i, 0), ch_tiles(A, head.r, head.i, 1));
    ch_part(head, P.lo, P.hi, n, first, last);
    cut.more = first > 0 && last > first;
    n = max(ch_tiles(A, tail.r, tail.i, 0), ch_tiles(A, tail.r, tail.i, 1));
    ch_part(tail, P.lo, P.hi, n, first, last);
    cut.last = -1;
    if (first == 0 && last > 0 && last < n) {
        const int64_t end = tail.start + tail.cost - 1;       // and the range that holds it
        int k = (int)min(end / max(P.all / P.ranges, (int64_t)1), (int64_t)P.ranges - 1);
        while (k + 1 < P.ranges && ch_bound(P.all, P.ranges, k + 1) <= end) ++k;
        while (k > 0 && ch_bound(P.all, P.ranges, k) > end) --k;
        cut.last = k;
    }
    cut.row = tail.r.a;
    cut.tok0 = tail.i * 2 * A.tq;
    cut.n = tail.r.n;
    cut.g = tail.g;
    return cut;
}

// ------------------------------------------------------------------ softmax
// 32 bytes, a whole sector, from one thread: a warp's threads hold a row each.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// One arrival for the warp, after what all its threads did.  (32 of them are made one by one.)
__device__ __forceinline__ void warp_arrive(uint64_t& bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
}
// A barrier of 128 threads, and whether any of them asked for `x`.  One warp waits for an mbarrier and the others here:
// every warp that waits at an mbarrier is woken by others' arrivals, and takes issue slots.
__device__ __forceinline__ bool group_any(int id, bool x) {
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred.aligned q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(any)
        : "r"((uint32_t)x), "r"(id)
        : "memory");
    return any != 0;
}

// What the sum l of a row's exponentials counts in, 2^(m - c).
struct ChUnit {
    float m, c;
    __device__ __forceinline__ bool above(const ChUnit& o) const { return m - o.m > c - o.c; }
    __device__ __forceinline__ float in(const ChUnit& o) const { return ex2((m - o.m) - (c - o.c)); }      // 1 of this in units of `o`
    __device__ __forceinline__ ChUnit with(float to) const { return {to, floorf(to - m + c)}; }            // the next above with this m
};

__device__ __forceinline__ bool ch_big(float m) { return fabsf(m) >= CH_BIG && fabsf(m) < INFINITY; }
// A key's factor from product to score.  (A masked score times zero would be NaN.)
template <bool FP8>
__device__ __forceinline__ float ch_scale(float q_scale, float k_scale) { return FP8 ? fmaxf(k_scale * q_scale, 1.2e-38f) : q_scale; }
// What few tiles of scores need, before their weights.  l and c before the tile, and by how much m has risen; returns l with the
// tile's share, and c, where scales are far apart.  For d 128 a function of its own, as the others' code has to fit
// the instruction caches (8192 tokens in e4m3 478 us, 499 with it inside); for d 64 it is faster inside (417 us against 470).
template <bool FP8>
__device__ __forceinline__ float2 ch_rare_tile(const ChShared& sh, uint32_t S, uint32_t slot, float q_scale, bool far_scales, float m, float l, float rise, float c) {
    constexpr float CH_BIAS = CH_BIAS_OF<FP8>;
    // Large scores: m is the maximum of rounded ones, and m's rounding alone would take exp2(x scale - m) out of its range.
    // They become what, times the scale, is each one's distance from m.
    const bool big = ch_big(m);
    const float b = m == -INFINITY ? 0.f : CH_BIAS - (big ? 0.f : m);
    // Scales far apart: a weight times 2^c / v_scale may pass fp32's range, or the weight be 0 where its share of l is not.
    // There shares are exponentials of their own, and c follows down to the page that leads among them.  What leads m may be a
    // larger scale alone, and what came before still be most of l: l does not shrink as m rises, but c does rise; and an l that
    // has become small is counted in a smaller unit, so that c is no lower than it has to be.
    if (far_scales) {
        const float whole = floorf(rise);
        const int up = l != 0.f && l < 0x1p-32f ? 127 - (int)(__float_as_uint(l) >> 23) : 0;
        c = l == 0.f ? CH_TOP_C : c + whole + (float)up;
        l = l * ex2(whole - rise) * __uint_as_float((uint32_t)(up + 127) << 23);
    }
#pragma unroll 1
    for (int g = 0; g < 16; ++g) {
        uint32_t x[8];
        tmem_ld8(S + 8 * g, x);
        tmem_wait_ld();
        const float v = FP8 ? sh.v_log[slot][g / 2] : 0.f, scale = ch_scale<FP8>(q_scale, sh.k_scale[slot][g / 2]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = __uint_as_float(x[e]), z = FP8 ? fmaf(y, scale, v) : __fmul_rn(y, scale);
            x[e] = __float_as_uint(big ? __fdividef(__fsub_rn(z, m) - v, scale) : y);
        }
        tmem_st8(S + 8 * g, x);
        if (FP8 && far_scales) {
            float y[8], first = -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; ++e) first = fmaxf(first, y[e] = fmaf(__uint_as_float(x[e]), scale, b + v));
            const bool seen = first != -INFINITY;
            const float low = seen ? fminf(c, floorf(v + CH_BIAS - first)) : c, by = seen ? low - v : -INFINITY;
            l *= ex2(low - c);
            c = low;               // no share is above 2^6
#pragma unroll
            for (int e = 0; e < 8; ++e) l += ex2(y[e] + by);
        }
    }
    tmem_wait_st();
    return make_float2(l, c);
}
template <bool FP8>
__device__ __noinline__ float2 ch_rare_call(const ChShared& sh, uint32_t S, uint32_t slot, float q_scale, bool far_scales, float m, float l, float rise, float c) {
    return ch_rare_tile<FP8>(sh, S, slot, q_scale, far_scales, m, l, rise, c);
}

// The softmax of one tile of an item: a thread owns a row; it sees its request's keys [0, limit).  False: a wait gave up.
template <int D, bool FP8>
__device__ __forceinline__ bool ch_softmax(ChShared& sh, const ChunkArgs& A, const ChunkItem& I, int t, uint32_t events, uint32_t keys, uint32_t& shares) {
    const uint32_t lanes = (uint32_t)(threadIdx.x & 96) << 16;          // this warp's quarter of the lanes
    const uint32_t S = sh.tmem + 128 * t + lanes, O = sh.tmem + 256 + D * t + lanes;
    const int row = threadIdx.x & 127, tl = row / A.r, head = row - tl * A.r;
    const int tok = I.tok0 + (I.dual ? 0 : t * A.tq) + tl;
    const bool real = tl < A.tq && tok < I.nq;
    const bool any = __any_sync(0xffffffffu, real);
    const int n_tiles = I.n(t);
    // a row that is none may see anything
    const int limit = real ? (int)min(max((int64_t)tok + 1 + (I.len - I.nq), (int64_t)0), (int64_t)I.len) - I.first * CH_KEYS : INT32_MAX;
    // log2 units.  Next to e4m3 pages m is the maximum of the scores times their v_scale.  l is in units of 2^(m - c) (and of 2^-6, as the weights);
    // c is 0 next to bf16.
    constexpr float CH_BIAS = CH_BIAS_OF<FP8>;
    float m = -INFINITY, l = 0.f, c = 0.f;
    float pass = -INFINITY, b = 0.f;                                    // a score beyond this raises m; what is added to a score
    float q_scale = A.scale_log2;
    int q_exp = 0;
    if (FP8 && real) q_exp = A.q_exp[(I.row + tok) * A.hq + I.g * A.r + head];
    const int step = I.dual ? 2 : 1;                                    // of the item's tiles of keys, from tile j on
    int j = I.dual ? t : 0;
    for (int i = 0; i < n_tiles; ++i, j += step) {
        const uint32_t slot = (keys + j) % CH_SCALES;
        bool ok = true;
        if ((threadIdx.x & 96) == 0)           // the group's first warp
            ok = ch_event(sh, A, t, events + (step == 2 ? 2 * i : i)) && ch_wait(sh, A, sh.sc_full[slot], (keys + j) / CH_SCALES);
        if (group_any(1 + t, !ok)) return false;
        if (!any) {                // no rows in this warp: nothing reads what its lanes of P and O hold
            for (int h = 0; h < 2; ++h) warp_arrive(sh.p_full[t][h]);
            continue;
        }
        tc_fence_after();
        const uint2 bads = sh.bad[slot];
        if (FP8 && i == 0) c = __uint_as_float(bads.y);
        if (FP8 && i == 0) q_scale = q_exp == CH_NAN ? 0.f : __uint_as_float((uint32_t)(127 - q_exp) << 23) * A.scale_log2;
        const uint32_t bad = bads.x & 0xFF;
        const bool far_scales = FP8 && bads.x >= CH_FAR;
        const int rem = min(limit - j * CH_KEYS, CH_KEYS);
        const bool edge = bad || __any_sync(0xffffffffu, rem < CH_KEYS);
        auto scale_of = [&](float k_scale) { return ch_scale<FP8>(q_scale, k_scale); };
        auto top_of = [](const uint32_t* x) {
            float u = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])), v = fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3]));
#pragma unroll
            for (int e = 4; e < 16; e += 4) {
                u = max3(u, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                v = max3(v, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
            }
            return fmaxf(u, v);
        };
        // 16 scores to weights, two to a word.
        auto weights = [&](const uint32_t* x, uint32_t* p, float scale, float b, uint64_t (&sum)[2]) {
            const uint64_t scale2 = pack2(scale, scale), b2 = pack2(b, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float u, v;
                unpack2(fma2(pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale2, b2), u, v);
                u = ex2(u);
                v = ex2(v);
                sum[e & 1] = add2(sum[e & 1], pack2(u, v));
                if (FP8) {
                    const __half2 y = __floats2half2_rn(u, v);
                    p[e] = *reinterpret_cast<const uint32_t*>(&y);
                } else {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(u, v);
                    p[e] = *reinterpret_cast<const uint32_t*>(&y);
                }
            }
        };
        // Keys that a row does not see, at an item's end: hidden in tensor memory.
        if (edge) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t y[32];
                tmem_ld32(S + 32 * c, y);
                tmem_wait_ld();
                const uint32_t seen = rem >= 32 * c + 32 ? ~0u : rem <= 32 * c ? 0u : (1u << (rem - 32 * c)) - 1;
                const uint32_t keep = seen & ~((bad >> 2 * c & 1 ? 0xFFFFu : 0u) | (bad >> 2 * c & 2 ? 0xFFFF0000u : 0u));
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!(keep >> e & 1)) y[e] = 0xFF800000u;           // -inf
                tmem_st32(S + 32 * c, y);
            }
            tmem_wait_st();
        }
        // Half of the keys at a time, in loops that stay loops: what two warps of a scheduler, the products' and the widening
        // one run all the time has to fit its instruction cache.
        uint32_t x[64];
        float top = -INFINITY;
#pragma unroll 1
        for (int h = 1; h >= 0; --h) {
            tmem_ld32(S + 64 * h, x);
            tmem_ld32(S + 64 * h + 32, x + 32);
            tmem_wait_ld();
            if (FP8) {
                const float4 k = *reinterpret_cast<const float4*>(&sh.k_scale[slot][4 * h]), v = *reinterpret_cast<const float4*>(&sh.v_log[slot][4 * h]);
                const float ks[4] = {k.x, k.y, k.z, k.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int g = 0; g < 4; ++g) top = fmaxf(top, fmaf(top_of(x + 16 * g), scale_of(ks[g]), vs[g]));
            } else {
#pragma unroll
                for (int g = 0; g < 4; g += 2) top = max3(top, top_of(x + 16 * g), top_of(x + 16 * g + 16));
            }
        }
        if (!FP8) top *= q_scale;
        if (far_scales || __any_sync(0xffffffffu, real && top > pass)) {
            const float to = fmaxf(m, top);
            const float f = m == -INFINITY ? 0.f : ex2(m - to);
            const float l_before = l, was = m;
            l *= f;
            m = to;
            pass = fabsf(m) < CH_BIG ? m + CH_RAISE : -INFINITY;
            b = fabsf(m) < CH_BIG ? CH_BIAS - m : m == -INFINITY ? 0.f : m == INFINITY ? __uint_as_float(0x7FC00000u) : CH_BIAS;
            if (i > 0) {           // these scores are complete: so is the value product that was issued before them
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32];
                    tmem_ld32(O + x, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st32(O + x, o);
                }
            }
            if (far_scales || __any_sync(0xffffffffu, real && ch_big(m))) {
                const float rise = l_before == 0.f ? 0.f : to - was;
                const float2 lc = D == 64 ? ch_rare_tile<FP8>(sh, S, slot, q_scale, far_scales, m, l_before, rise, c)
                                          : ch_rare_call<FP8>(sh, S, slot, q_scale, far_scales, m, l_before, rise, c);
                if (far_scales) {
                    l = lc.x;
                    c = lc.y;
                }
                tmem_ld32(S, x);
                tmem_ld32(S + 32, x + 32);
                tmem_wait_ld();
            }
        }
        uint64_t sum[2] = {0ull, 0ull};
        float total = 0.f;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {          // (the first half is still there)
            uint32_t p[32];
            const float4 k = *reinterpret_cast<const float4*>(&sh.k_scale[slot][4 * h]), v = *reinterpret_cast<const float4*>(&sh.v_log[slot][4 * h]);
            const float4 share = *reinterpret_cast<const float4*>(&sh.v_share[slot][4 * h]);
            const float ks[4] = {k.x, k.y, k.z, k.w}, vs[4] = {v.x, v.y, v.z, v.w}, shares[4] = {share.x, share.y, share.z, share.w};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (FP8) {
                    sum[0] = sum[1] = 0ull;
                    weights(x + 16 * g, p + 8 * g, scale_of(ks[g]), b + vs[g], sum);
                    float s0, s1;
                    unpack2(add2(sum[0], sum[1]), s0, s1);
                    total = fmaf(s0 + s1, shares[g], total);
                } else {
                    weights(x + 16 * g, p + 8 * g, q_scale, b, sum);
                }
            }
            if (h == 0) {
                tmem_ld32(S + 64, x);
                tmem_ld32(S + 96, x + 32);
            }
            tmem_st32(S + 32 * h, p);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(sh.p_full[t][h]);      // the value product may begin on half of the keys
            tmem_wait_ld();
        }
        if (!FP8) {
            float s0, s1;
            unpack2(add2(sum[0], sum[1]), s0, s1);
            total = s0 + s1;
        }
        l += total;
    }
    if (FP8) {                     // for all but extreme scales c is 0 from here on
        l *= fabsf(c) <= CH_NEAR ? ex2(-c) : 1.f;
        c = fabsf(c) <= CH_NEAR || l == 0.f ? 0.f : c;
    }
    if (q_exp == CH_NAN && n_tiles > 0) l = __uint_as_float(0x7FC00000u);
    if (n_tiles > 0) {
        bool ok = true;
        if ((threadIdx.x & 96) == 0) ok = ch_event(sh, A, t, events + I.event(n_tiles - 1, 1));
        if (group_any(1 + t, !ok)) return false;
        tc_fence_after();
    }
    // A dual item's halves: this thread writes half of the row's values, from both.  (The fences about the exchange order the other
    // half's products, which its threads have waited for, before this one's loads of them.)
    const bool both = I.dual && I.n1 > 0;
    float w0 = t == 0 ? 1.f : 0.f, w1 = 1.f - w0;              // weights of the tiles' sums
    float lse = 0.f;               // log2
    // 2^c / l, but for a power of two that would take it out of fp32's range, which is left in c.
    auto inverse = [&]() {
        if (!FP8 || c == 0.f) return l != 0.f ? 1.f / l : 0.f;
        const int e = min((int)(__float_as_uint(l) >> 23 & 255) - 127, 126);
        const float all = c - (float)e, here = fminf(fmaxf(all, -64.f), 64.f);
        c = all - here;
        return 1.f / (l * __uint_as_float((uint32_t)(127 - e) << 23)) * ex2(here);
    };
    if (both) {
        bool ok = true;
        if (t == 1) {
            sh.share[row] = make_float2(m, l);
            if (FP8) sh.share_c[row] = (int16_t)c;
            tc_fence_before();
            warp_arrive(sh.ml_there);
            if ((threadIdx.x & 96) == 0) ok = ch_wait(sh, A, sh.weights_there, shares);
            if (group_any(2, !ok)) return false;
            tc_fence_after();
            const float2 x = sh.share[row];
            w0 = x.x;
            w1 = x.y;
            if (FP8) c = sh.share_c[row];
        } else {
            if ((threadIdx.x & 96) == 0) ok = ch_wait(sh, A, sh.ml_there, shares);
            if (group_any(1, !ok)) return false;
            tc_fence_after();
            const float2 x = sh.share[row];
            const float to = fmaxf(l != 0.f ? m : -INFINITY, x.y != 0.f ? x.x : -INFINITY);
            w0 = l != 0.f ? ex2(m - to) : 0.f;                 // one that saw nothing has weight 0
            w1 = x.y != 0.f ? ex2(x.x - to) : 0.f;
            const float c1 = FP8 ? (float)sh.share_c[row] : 0.f;
            if (FP8 && __any_sync(0xffffffffu, c != 0.f || c1 != 0.f)) {
                const ChUnit u{m, c}, u1{x.x, c1};
                const bool above = l == 0.f || (x.y != 0.f && u1.above(u));
                const ChUnit sum = ChUnit{above ? u1.m : u.m, above ? u1.c : u.c}.with(to);
                l = (l != 0.f ? u.in(sum) * l : 0.f) + (x.y != 0.f ? u1.in(sum) * x.y : 0.f);
                c = l != 0.f ? sum.c : 0.f;
            } else {
                l = (l != 0.f ? w0 * l : 0.f) + (x.y != 0.f ? w1 * x.y : 0.f);
            }
            m = to;
            if (I.part < 0) {
                lse = l == 0.f ? -INFINITY : m - c + log2f(l) - CH_BIAS;
                const float inv = inverse();
                w0 *= inv;
                w1 *= inv;
                if (FP8) sh.share_c[row] = (int16_t)c;
            }
            sh.share[row] = make_float2(w0, w1);
            tc_fence_before();
            warp_arrive(sh.weights_there);
        }
        ++shares;
    } else if (I.part < 0) {
        lse = l == 0.f ? -INFINITY : m - c + log2f(l) - CH_BIAS;
        const float inv = inverse();
        w0 *= inv;
        w1 *= inv;
    }
    if (I.dual && !both && t == 1) return true;
    const int tile = I.dual ? 0 : t, col0 = both ? t * (D / 2) : 0, cols = both ? D / 2 : D;
    const bool some = both || n_tiles > 0;
    const int64_t at = I.part >= 0 ? (int64_t)I.part * A.tiles + tile : 0, out = (I.row + tok) * A.hq + I.g * A.r + head;
    const uint32_t O0 = sh.tmem + 256 + lanes, O1 = O0 + D;
    const float rest = FP8 && I.part < 0 ? ex2(c) : 1.f;
    const uint64_t rest2 = pack2(rest, rest);
    if (any)
#pragma unroll 1
        for (int x = col0; x < col0 + cols; x += 32) {
            uint32_t o[32];
            if (some) {
                tmem_ld32((both || t == 0 ? O0 : O1) + x, o);
                tmem_wait_ld();
                // a row that saw nothing is zero, whatever its lane of tensor memory holds
                const float f = both || t == 0 ? w0 : w1;
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = f != 0.f ? __float_as_uint(__uint_as_float(o[i]) * f) : 0u;
                if (both) {
                    uint32_t o1[32];
                    tmem_ld32(O1 + x, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (w1 != 0.f) o[i] = __float_as_uint(fmaf(w1, __uint_as_float(o1[i]), __uint_as_float(o[i])));
                }
                if (FP8)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float y, z;
                        unpack2(mul2(pack2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), rest2), y, z);
                        o[i] = __float_as_uint(y);
                        o[i + 1] = __float_as_uint(z);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0u;
            }
            if (I.part >= 0) {     // a part of the item, for the join
                float4* to = reinterpret_cast<float4*>(A.part_o) + (at * (D / 4) + x / 4) * CH_ROWS + row;
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (real)
                        to[i / 4 * CH_ROWS] = make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
            } else {
                uint16_t* to = A.o + out * D + x;
#pragma unroll
                for (int i = 0; i < 32; i += 16) {
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[i + 2 * e]), __uint_as_float(o[i + 2 * e + 1]));
                        y[e] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                    if (!real) continue;
                    if (A.wide) {
                        st_global_32(to + i, y);
                    } else {
                        *reinterpret_cast<uint4*>(to + i) = make_uint4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<uint4*>(to + i + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                    }
                }
            }
        }
    if (both) {                    // the next item's value products may go over these sums
        tc_fence_before();
        warp_arrive(sh.o_read);
    }
    if (real && (!both || t == 0)) {
        if (I.part >= 0) {
            if constexpr (FP8) reinterpret_cast<float4*>(A.part_ml)[at * CH_ROWS + row] = make_float4(m, l, c, 0.f);
            else reinterpret_cast<float2*>(A.part_ml)[at * CH_ROWS + row] = make_float2(m, l);
        } else if (A.lse) {
            A.lse[out] = lse * 0.6931471805599453f;
        }
    }
    return true;
}

// ------------------------------------------------------------------ q and V of 8-bit pages
// The launch before the others, next to e4m3 pages: the rows of q as sums of two e4m3 pieces, q8 [2][rows][D], times
// 2^q_exp[row]; D / 16 threads to a row.
constexpr int CS_THREADS = 256;
template <int D>
__global__ void __launch_bounds__(CS_THREADS) paged_chunk_split_kernel(const uint16_t* q, int64_t q_stride, int hq, int64_t rows, uint8_t* q8, int8_t* q_exp) {
    constexpr int LANES = D / 16;
    grid_wait();
    grid_launch_next();
    const int64_t i = (int64_t)blockIdx.x * CS_THREADS + threadIdx.x, row = i / LANES;
    const int c = (int)(i % LANES);
    const bool in = row < rows;
    uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (in) {
        const int64_t tok = row / hq;
        const uint4* from = reinterpret_cast<const uint4*>(q + tok * q_stride + (row - tok * hq) * D) + 2 * c;
        v[0] = __ldg(from);
        v[1] = __ldg(from + 1);
    }
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t top2 = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top2 = __vmaxu2(top2, w[k] & 0x7FFF7FFFu);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, o));
    const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);     // the largest magnitude's bits
    const bool finite = top < 0x7F80u;
    const int e = min(7 - ((int)(top >> 7) - 127), 120);      // 2^7 <= largest * 2^e < 2^8
    const float up = finite ? __uint_as_float((uint32_t)(e + 127) << 23) : 0.f;
    uint32_t a[4], b[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t x2 = finite ? w[k] : 0u;
        const float x = __uint_as_float(x2 << 16) * up, y = __uint_as_float(x2 & 0xFFFF0000u) * up;
        const uint16_t hi = f32x2_to_e4m3x2(x, y);
        const uint32_t f = e4m3x2_to_f16x2(hi);
        const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&f));
        const uint16_t lo = f32x2_to_e4m3x2(x - got.x, y - got.y);
        if (k & 1) { a[k / 2] |= (uint32_t)hi << 16; b[k / 2] |= (uint32_t)lo << 16; }
        else { a[k / 2] = hi; b[k / 2] = lo; }
    }
    if (!in) return;
    *reinterpret_cast<uint4*>(q8 + row * D + 16 * c) = make_uint4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<uint4*>(q8 + (rows + row) * D + 16 * c) = make_uint4(b[0], b[1], b[2], b[3]);
    if (c == 0) q_exp[row] = (int8_t)(finite ? e : CH_NAN);
}

// A tile of V from its codes to f16, by 128 threads; rows from `have` on become zero, as a weight of zero does not silence the
// NaN that may lie there.
template <int D>
__device__ __forceinline__ void ch_widen_v(const uint8_t* from, uint8_t* to, int have) {
    constexpr int CH = D / 16;
    const int t = threadIdx.x & 127, row0 = t / CH, c = t % CH;
    // Rows of a thread are 128 / CH apart, a multiple of 8: their swizzles are alike.
    const uint8_t* a = from + row0 * D + (D == 128 ? c ^ (row0 & 7) : c ^ (row0 >> 1 & 3)) * 16;
    uint8_t* b = to + (c / 4) * CH_BLOCK + row0 * 128;
    const int x0 = ((c % 4 * 2) ^ (row0 & 7)) * 16, x1 = ((c % 4 * 2 + 1) ^ (row0 & 7)) * 16;
    uint4 v[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) v[k] = *reinterpret_cast<const uint4*>(a + k * (128 / CH) * D);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = e4m3x2_to_f16x2((uint16_t)(w[i / 2] >> (i & 1) * 16));
        if (row0 + k * (128 / CH) >= have)
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = 0u;
        // Eight lanes hold a row; half of them begin with the second chunk, so that the eight meet all banks.
        uint8_t* to_row = b + k * (128 / CH) * 128;
        const bool second = c / 4 & 1;
        const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
        *reinterpret_cast<uint4*>(to_row + (second ? x1 : x0)) = second ? hi : lo;
        *reinterpret_cast<uint4*>(to_row + (second ? x0 : x1)) = second ? lo : hi;
    }
}

// ------------------------------------------------------------------ the kernel
template <int D, bool FP8>
__global__ void __launch_bounds__(ChShape<D, FP8>::THREADS, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ ChunkArgs A) {
    using P = ChShape<D, FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];           // the tiles, then ChShared
    ChShared& sh = *reinterpret_cast<ChShared*>(smem + P::TILES);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t K0 = 2 * P::Q, V0 = K0 + P::KS * P::TILE, WIDE0 = V0 + P::VS * P::TILE;
    if (tid == 0) {
        tensor_map_prefetch(&map_q);
        tensor_map_prefetch(&map_k);
        tensor_map_prefetch(&map_v);
        for (int i = 0; i < P::KS; ++i) mbar_init(smem_u32(&sh.k_full[i]), 1);
        for (int i = 0; i < P::VS; ++i) mbar_init(smem_u32(&sh.v_full[i]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.raw_free[i]), 4);
        for (int i = 0; i < P::WIDES; ++i) mbar_init(smem_u32(&sh.wide_full[i]), 4);
        mbar_init(smem_u32(&sh.ml_there), 4);
        mbar_init(smem_u32(&sh.weights_there), 4);
        mbar_init(smem_u32(&sh.o_read), 8);
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&sh.q_full[t]), 1);
            for (int i = 0; i < CH_EVENTS; ++i) mbar_init(smem_u32(&sh.event[t][i]), 1);
            for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.p_full[t][i]), 4);
            mbar_init(smem_u32(&sh.turn[t]), 1);
            mbar_init(smem_u32(&sh.drain[t]), 1);
        }
        mbar_init(smem_u32(&sh.v_tail), 1);
        for (int i = 0; i < CH_ITEMS; ++i) {
            mbar_init(smem_u32(&sh.item_full[i]), 1);
            mbar_init(smem_u32(&sh.item_free[i]), FP8 ? 14 : 11);
        }
        for (int i = 0; i < CH_SCALES; ++i) mbar_init(smem_u32(&sh.sc_full[i]), 1);
        sh.abort = sh.k_issued = sh.v_issued = sh.tail_open = sh.tail_phase = sh.q_issued[0] = sh.q_issued[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    grid_wait();
    ChPlan plan;
    const bool aligned = (base & 1023) == 0;   // as declared; the swizzled tiles would be elsewhere
    if (!aligned && tid == 0 && A.status) atomicOr(A.status, KVO_DEV_TIMEOUT);
    if (!aligned || !ch_plan<P::THREADS>(sh, A, plan)) {
        if (tid == 0) {
            ChunkCut cut{};
            cut.last = -1;
            A.cut[blockIdx.x] = cut;
        }
        return;
    }
    if (warp == 8) tmem_alloc(smem_u32(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    // The next item, once the walking warp has written it.
    auto next_item = [&](uint32_t k, ChunkItem& I) {
        if (!ch_wait(sh, A, sh.item_full[k % CH_ITEMS], k / CH_ITEMS)) return false;
        I = sh.item[k % CH_ITEMS];
        return true;
    };
    // Of the item's tiles j .. j + 3, the (lane % 8)-th 16 keys of tile j + lane / 8: the first of them, and their page, an entry
    // of the table that may be anything and is not looked at here (it is on its way); -1 behind the last key.
    auto key_of = [&](const ChunkItem& I, int j) { return (int64_t)(I.first + j + (lane >> 3)) * CH_KEYS + 16 * (lane & 7); };
    auto page_of = [&](const ChunkItem& I, int j) {
        const int64_t key = key_of(I, j);
        return key < I.len ? __ldg(A.table + (int64_t)I.b * A.max_pages + (key >> A.shift)) : -1;
    };
    // Whole warp: asks for a tile of K or V, a box to a lane: its page's rows in the pool, or, where there is no such page,
    // what lies behind the last (zeros).
    auto load_tile = [&](const CUtensorMap* map, const ChunkItem& I, int page, int j, uint32_t at, uint32_t bar, int number) {
        constexpr int ROW = D * (FP8 ? 1 : 2), BOXES = ROW > 128 ? ROW / 128 : 1, BOX = ROW > 128 ? 128 : ROW;
        const int from = __shfl_sync(0xffffffffu, page, (j & 3) * 8 + lane / BOXES * (A.page / 16) & 31);
        const int y = from < 0 ? A.n_pages * A.hkv * A.page : (from * A.hkv + I.g) * A.page;
        if (lane < CH_KEYS / A.page * BOXES && number != A.skip)
            tma_load_2d(base + at + (lane % BOXES) * CH_BLOCK + lane / BOXES * A.page * BOX, map, (lane % BOXES) * (FP8 ? 128 : 64), y, bar);
    };
    auto event_wait = [&](int t, uint32_t e) { return e == ~0u || ch_event(sh, A, t, e); };
    auto free_item = [&](uint32_t k) { mbar_arrive(smem_u32(&sh.item_free[k % CH_ITEMS])); };

    if (warp >= 8) {
        regs_dec<P::REGS_OTHER>();
        if (warp == 9) {
            // ------------------------------------------------ items, loads
            ChWalk walk = ch_locate(A, sh.found[0], ch_request(A, sh.found[0]), sh.at[0], plan.lo);
            int high = sh.high[0];
            const int64_t lo = plan.lo, hi = plan.hi;
            if (FP8) {
                if (lane == 0) A.cut[blockIdx.x] = ch_cut(sh, A, plan, walk);        // before anything that may give up: the join follows it
                __syncwarp();
            }
            bool ok = true;
            uint32_t k = 0, tiles = 0, v_issued = 0;
            uint32_t events[2] = {0, 0}, q_issued[2] = {0, 0};
            uint32_t q_free[2] = {~0u, ~0u};            // the event after which a tile's q may be overwritten
            uint32_t e0 = ~0u, e1 = ~0u;                // of stage `lane`: the events that free it
            while (ok) {
                int first, last;
                const int all0 = ch_tiles(A, walk.r, walk.i, 0), all1 = ch_tiles(A, walk.r, walk.i, 1), n_item = max(all0, all1);
                ch_part(walk, lo, hi, n_item, first, last);
                if (n_item ? last > first : walk.start >= lo) {
                    ChunkItem I;
                    I.row = walk.r.a;
                    I.first = first;
                    I.dual = walk.r.n - walk.i * 2 * A.tq <= A.tq;
                    I.tiles = last - first;
                    I.n0 = I.dual ? (I.tiles + 1) / 2 : min(max(all0 - first, 0), I.tiles);
                    I.n1 = I.dual ? I.tiles / 2 : min(max(all1 - first, 0), I.tiles);
                    I.b = walk.b;
                    I.g = walk.g;
                    I.tok0 = walk.i * 2 * A.tq;
                    I.nq = walk.r.n;
                    I.len = walk.r.len;
                    I.part = first == 0 && last == n_item ? -1 : 2 * (int)blockIdx.x + (first == 0);
                    if (k >= CH_ITEMS) ok = ch_wait(sh, A, sh.item_free[k % CH_ITEMS], k / CH_ITEMS - 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    if (lane == 0) {
                        sh.item[k % CH_ITEMS] = I;
                        mbar_arrive(smem_u32(&sh.item_full[k % CH_ITEMS]));
                    }
                    ++k;
                    int page = 0, page_next = page_of(I, 0);
                    bool bad = false;
                    float ks = 0.f, vs = 0.f, v_log = 0.f, v_share = 0.f, v_first = 0.f;
                    uint32_t far = 0;
                    for (int j = 0; ok && j < I.tiles; ++j, ++tiles) {
                        if ((j & 3) == 0) {
                            page = page_next;
                            if (j + 4 < I.tiles) page_next = page_of(I, j + 4);
                            const bool in = key_of(I, j) < I.len;
                            bad = in && (page < 0 || page >= A.n_pages);
                            if (bad && j + (lane >> 3) < I.tiles && A.status) atomicOr(A.status, KVO_DEV_BAD_BLOCK_ID);
                            if (bad || !in) page = -1;
                            if constexpr (FP8) {
                                ks = page < 0 ? 1.f : __ldg(A.k_scale + (int64_t)page * A.hkv + I.g);
                                vs = page < 0 ? 1.f : __ldg(A.v_scale + (int64_t)page * A.hkv + I.g);
                            }
                        }
                        const uint32_t bads = __ballot_sync(0xffffffffu, bad) >> (j & 3) * 8 & 0xFF;
                        const int st = tiles % P::KS, sc = tiles % CH_SCALES;
                        if (tiles >= P::KS) {
                            ok = event_wait(0, __shfl_sync(0xffffffffu, e0, st));
                            ok = event_wait(1, __shfl_sync(0xffffffffu, e1, st)) && ok;
                            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                        }
                        if (lane == 0) mbar_expect_tx(smem_u32(&sh.k_full[st]), P::TILE);
                        __syncwarp();
                        load_tile(&map_k, I, page, j, K0 + st * P::TILE, smem_u32(&sh.k_full[st]), 2 * tiles);
                        if (lane == st) {
                            const int i = I.dual ? j >> 1 : j;
                            e0 = (I.dual ? !(j & 1) : j < I.n0) ? events[0] + I.event(i, 0) : ~0u;
                            e1 = (I.dual ? j & 1 : j < I.n1) ? events[1] + I.event(i, 0) : ~0u;
                        }
                        if (j == 0)
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                if (I.n(t) == 0 || !ok) continue;
                                ok = event_wait(t, q_free[t]);
                                ok = __all_sync(0xffffffffu, ok);
                                if (lane == 0 && ok) {
                                    mbar_expect_tx(smem_u32(&sh.q_full[t]), (uint32_t)(2 * D * A.r * A.tq));
                                    const int tok = (int)I.row + I.tok0 + (I.dual ? 0 : t * A.tq);
                                    for (int x = 0; x < (FP8 ? 2 : D / 64); ++x)         // the pieces, or 64 values of d
                                        tma_load_3d(base + t * P::Q + x * (FP8 ? CH_ROWS * D : CH_BLOCK), &map_q, FP8 ? 0 : 64 * x, I.g * A.r,
                                                    tok + (FP8 ? x * (int)A.total : 0), smem_u32(&sh.q_full[t]));
                                }
                                q_issued[t] += ok;
                            }
                        // What the softmax has to know of the tile, while its keys are on their way.
                        if constexpr (FP8) {
                            if ((j & 3) == 0) {
                                const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
                                v_log = vs == 0.f ? CH_NO_SCALE : log2f(vs);
                                if (j == 0) v_first = there ? rintf(__shfl_sync(0xffffffffu, v_log, __ffs((int)there) - 1)) : 0.f;
                                if (page < 0) v_log = v_first;          // (nothing is seen there)
                                far |= __any_sync(0xffffffffu, !(fabsf(v_log - v_first) <= CH_SPREAD)) ? CH_FAR : 0u;
                                v_share = far ? 0.f : exp2f(v_first - v_log);
                            }
                            if (lane >> 3 == (j & 3)) {
                                sh.k_scale[sc][lane & 7] = ks;
                                sh.v_log[sc][lane & 7] = v_log;
                                sh.v_share[sc][lane & 7] = v_share;
                            }
                        }
                        if (lane == 0) sh.bad[sc] = make_uint2(bads | far, __float_as_uint(v_first));
                        warp_arrive(sh.sc_full[sc]);
                        if constexpr (FP8) {
                            const int sv = tiles % P::VS;
                            if (ok && tiles >= P::VS) ok = ch_wait(sh, A, sh.raw_free[sv], tiles / P::VS - 1);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) { ++tiles; break; }
                            if (lane == 0) mbar_expect_tx(smem_u32(&sh.v_full[sv]), P::TILE);
                            __syncwarp();
                            load_tile(&map_v, I, page, j, V0 + sv * P::TILE, smem_u32(&sh.v_full[sv]), 2 * tiles + 1);
                            v_issued = tiles + 1;
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (I.n(t)) {
                            q_free[t] = events[t] + I.event(I.n(t) - 1, 0);
                            events[t] += I.events(t);
                        }
                }
                walk.start += walk.cost;
                if (!ok || walk.start >= hi) break;
                if (++walk.g == A.hkv) {
                    walk.g = 0;
                    if (++walk.i == ch_blocks(A, walk.r)) {
                        walk.i = 0;
                        do {                   // the range does not end here: there is another served request with new tokens
                            if (walk.r.served) high = max(high, walk.r.a + walk.r.n);
                            if (++walk.b >= A.batch) { ok = false; break; }
                            walk.r = ch_request(A, walk.b);
                            walk.r.served = walk.r.served && walk.r.a >= high;
                        } while (!walk.r.served || walk.r.n == 0);
                        if (!ok) { ok = true; break; }
                    }
                    walk.cost = ch_cost(A, walk.r, walk.i);
                }
            }
            if (ok && k >= CH_ITEMS) ok = ch_wait(sh, A, sh.item_free[k % CH_ITEMS], k / CH_ITEMS - 1);
            ok = __all_sync(0xffffffffu, ok);
            if (lane == 0) {
                if (ok) {
                    sh.item[k % CH_ITEMS].n0 = -1;
                    mbar_arrive(smem_u32(&sh.item_full[k % CH_ITEMS]));
                }
                sh.k_issued = tiles;
                if (FP8) sh.v_issued = v_issued;
            }
            // Where somebody gave up not all loads may have landed: the warp that issued them stays until they have, and
            // with it the CTA and its shared memory.  (`abort` is final only once all have left their waits: below.)
            __syncwarp();
            if (lane == 0) { sh.q_issued[0] = q_issued[0]; sh.q_issued[1] = q_issued[1]; }
        } else if (!FP8 && warp == 11) {
            if (lane == 0)                     // before anything that may give up: the join follows it
                A.cut[blockIdx.x] = ch_cut(sh, A, plan, ch_locate(A, sh.found[0], ch_request(A, sh.found[0]), sh.at[0], plan.lo));
            __syncwarp();
            // ------------------------------------------------ V, which waits for other things than K does
            bool ok = true, tail_open = false;
            uint32_t item = 0, tiles = 0, tail_phase = 0, events0 = 0, events1 = 0;
            uint32_t e0 = ~0u, e1 = ~0u;                // of stage `lane`: the events that free it
            while (ok) {
                ChunkItem I;
                ok = next_item(item, I);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok || I.n0 < 0) break;
                if (lane == 0) free_item(item);
                ++item;
                int page = 0, page_next = page_of(I, 0);
                for (int j = 0; j < I.tiles; ++j) {
                    if ((j & 3) == 0) {
                        page = page_next;
                        if (j + 4 < I.tiles) page_next = page_of(I, j + 4);
                        if (page < 0 || page >= A.n_pages) page = -1;
                    }
                    const int st = tiles % P::VS, key0 = (I.first + j) * CH_KEYS;
                    if (tiles >= P::VS) {
                        ok = event_wait(0, __shfl_sync(0xffffffffu, e0, st));
                        ok = event_wait(1, __shfl_sync(0xffffffffu, e1, st)) && ok;
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
                    // The last tile of a request runs into what lies behind it in its page.  Its keys are masked as scores, but a
                    // weight of zero does not silence a NaN or an infinity in V: those rows are cleared.
                    const bool tail = key0 + CH_KEYS > I.len;
                    const uint32_t bar = smem_u32(tail ? &sh.v_tail : &sh.v_full[st]);
                    if (lane == 0) mbar_expect_tx(bar, P::TILE);
                    __syncwarp();
                    load_tile(&map_v, I, page, j, V0 + st * P::TILE, bar, 2 * tiles + 1);
                    if (tail) {
                        tail_open = true;
                        ok = ch_wait(sh, A, sh.v_tail, tail_phase);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tail_open = false;
                        ++tail_phase;
                        for (int x = 0; x < D / 64; ++x)
                            for (uint32_t a = (I.len - key0) * 128 + lane * 16; a < CH_BLOCK; a += 512)
                                *reinterpret_cast<uint4*>(smem + V0 + st * P::TILE + x * CH_BLOCK + a) = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        warp_arrive(sh.v_full[st]);
                    }
                    if (lane == st) {
                        const int i = I.dual ? j >> 1 : j;
                        e0 = (I.dual ? !(j & 1) : j < I.n0) ? events0 + I.event(i, 1) : ~0u;
                        e1 = (I.dual ? j & 1 : j < I.n1) ? events1 + I.event(i, 1) : ~0u;
                    }
                    ++tiles;
                }
                events0 += I.events(0);
                events1 += I.events(1);
            }
            if (lane == 0) {
                sh.v_issued = tiles;
                sh.tail_open = tail_open;
                sh.tail_phase = tail_phase;
            }
        } else if ((warp == 8 || warp == 10) && elect_one()) {
            // ------------------------------------------------ matrix products of one tile
            // The tensor cores queue a few instructions only; with a thread of its own for each tile, one tile's waits and
            // commits pass while the other's products run.  They take turns, so that the tiles stay half a period apart.
            constexpr uint32_t ID_S = FP8 ? mma_desc_e4m3(CH_ROWS, CH_KEYS) : mma_desc(CH_ROWS, CH_KEYS, false);
            constexpr uint32_t ID_O = FP8 ? mma_desc_f16(CH_ROWS, D, true) : mma_desc(CH_ROWS, D, true);
            const int t = (warp - 8) >> 1;
            const uint32_t S = sh.tmem + 128 * t, O = sh.tmem + 256 + D * t;
            constexpr bool HALF = FP8 && D == 64;              // rows of 64 bytes
            const uint64_t q = HALF ? smem_desc64(base + t * P::Q) : smem_desc(base + t * P::Q, 16);
            const uint64_t k0 = HALF ? smem_desc64(base + K0) : smem_desc(base + K0, 16);
            const uint64_t v0 = smem_desc(base + (FP8 ? WIDE0 : V0), CH_BLOCK);
            uint32_t item = 0, events = 0, events_other = 0, weights = 0, qs = 0, turns = 0, tiles = 0, shares = 0;
            bool ok = true, behind = false, shared = false;
            while (true) {
                ChunkItem I;
                if (!next_item(item, I)) break;
                free_item(item++);
                if (I.n0 < 0) break;
                const int n_mine = I.n(t), n_other = I.n(t ^ 1);
                const bool turn = !I.dual && n_other > 0;
                // The i-th tile of keys of this tile of rows, counted over all items.
                auto at = [&](int i) { return tiles + (I.dual ? 2 * i + t : i); };
                auto keys_there = [&](int i) { return ch_wait(sh, A, sh.k_full[at(i) % P::KS], at(i) / P::KS); };
                auto values_there = [&](int i) {
                    return FP8 ? ch_wait(sh, A, sh.wide_full[at(i) % P::WIDES], at(i) / P::WIDES) : ch_wait(sh, A, sh.v_full[at(i) % P::VS], at(i) / P::VS);
                };
                if (n_mine > 0) {
                    // Tiles that only the other one used: their loads have landed once its products are complete (a barrier's
                    // parity tells phases apart only where none is passed over).
                    if (behind && !(ok = ch_event(sh, A, t ^ 1, events_other - 1))) break;
                    behind = false;
                    ok = ch_wait(sh, A, sh.q_full[t], qs++) && keys_there(0);
                    if (!ok) break;
                    for (int i = 0; i <= n_mine; ++i) {        // the value product of the tile before, then this one's scores
                        if (i > 0) {
                            if (!(ok = values_there(i - 1))) break;
                            if (i < n_mine && !(ok = keys_there(i))) break;
                            const uint64_t v = v0 + (uint64_t)(FP8 ? at(i - 1) % P::WIDES * (P::WIDE_BYTES >> 4) : at(i - 1) % P::VS * (P::TILE >> 4));
                            if (!(ok = ch_wait(sh, A, sh.p_full[t][0], weights))) break;
                            // Both halves of the last dual item have been read.
                            if (shared && !(ok = ch_wait(sh, A, sh.o_read, shares - 1))) break;
                            shared = false;
                            // The other tile's round before this one; that may be the last of an item before.  No phase is
                            // passed over.
                            const int x = t ? i - 1 : i - 2;
                            if (turn && x < n_other && turns + x != ~0u && !(ok = ch_wait(sh, A, sh.turn[t], turns + x))) break;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (h > 0 && !(ok = ch_wait(sh, A, sh.p_full[t][1], weights))) break;
                                tc_fence_after();
#pragma unroll
                                for (int e = 4 * h; e < 4 * h + 4; ++e) mma_ts(O, S + 8 * e, v + e * (2048 >> 4), ID_O, i > 1 || e > 0);
                            }
                            if (!ok) break;
                            ++weights;
                            // One commit for the next scores stands for the value product before them as well.
                            if (i == n_mine || I.dual) tc_commit(smem_u32(&sh.event[t][(events + I.event(i - 1, 1)) % CH_EVENTS]));
                        }
                        if (i == n_mine) {
                            if (turn) mbar_arrive(smem_u32(&sh.turn[t ^ 1]));
                            break;
                        }
                        tc_fence_after();
                        const uint64_t kd = k0 + (uint64_t)(at(i) % P::KS) * (P::TILE >> 4);
                        constexpr int STEPS = FP8 ? 2 * (D / 32) : D / 16;
#pragma unroll
                        for (int e = 0; e < STEPS; ++e) {
                            if (e == STEPS / 2 && turn && i > 0) mbar_arrive(smem_u32(&sh.turn[t ^ 1]));      // queued work covers the hand-over
                            if (FP8) {
                                constexpr int PER = D / 32;
                                mma_ss_e4m3(S, q + (e / PER) * (CH_ROWS * D >> 4) + (e % PER) * 2, kd + (e % PER) * 2, ID_S, e > 0);
                            } else {
                                const int off = (e >> 2) * (CH_BLOCK >> 4) + (e & 3) * 2;
                                mma_ss(S, q + off, kd + off, ID_S, e > 0);
                            }
                        }
                        tc_commit(smem_u32(&sh.event[t][(events + I.event(i, 0)) % CH_EVENTS]));
                    }
                    if (!ok) break;
                    events += I.events(t);
                    if (turn) turns += n_other;
                }
                if (I.dual ? n_other > 0 : n_other > n_mine) behind = true;
                events_other += I.events(t ^ 1);
                if (I.dual && I.n1 > 0) { shared = true; ++shares; }
                tiles += I.tiles;
            }
            // nothing of this CTA may be in flight when it leaves
            tc_commit(smem_u32(&sh.drain[t]));
            if (!mbar_wait_bounded(smem_u32(&sh.drain[t]), 0, A.wait_ns)) {
                *(volatile int*)&sh.abort = 1;
                if (A.status) atomicOr(A.status, KVO_DEV_TIMEOUT);
            }
        } else if (FP8 && warp >= 12) {
            // ------------------------------------------------ V of 8-bit pages
            if constexpr (FP8) {
                uint32_t item = 0, tiles = 0, events0 = 0, events1 = 0, e0 = ~0u, e1 = ~0u;         // of buffer `lane`: the events that free it
                bool ok = true;
                while (ok) {
                    ChunkItem I;
                    if (warp == 12) ok = ch_wait(sh, A, sh.item_full[item % CH_ITEMS], item / CH_ITEMS);
                    ok = !group_any(3, !ok);
                    if (!ok) break;
                    I = sh.item[item % CH_ITEMS];
                    __syncwarp();
                    if (lane == 0) free_item(item);
                    if (I.n0 < 0) break;
                    ++item;
                    for (int j = 0; j < I.tiles && ok; ++j) {
                        const int st = tiles % P::VS, w = tiles % P::WIDES;
                        const uint32_t free0 = __shfl_sync(0xffffffffu, e0, w), free1 = __shfl_sync(0xffffffffu, e1, w);
                        if (warp == 12) {
                            ok = ch_wait(sh, A, sh.v_full[st], tiles / P::VS);
                            if (ok && free0 != ~0u) ok = ch_event(sh, A, 0, free0);
                            if (ok && free1 != ~0u) ok = ch_event(sh, A, 1, free1);
                        }
                        ok = !group_any(3, !ok);
                        if (!ok) break;
                        ch_widen_v<D>(smem + V0 + st * P::TILE, smem + WIDE0 + w * P::WIDE_BYTES, I.len - (I.first + j) * CH_KEYS);
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(smem_u32(&sh.raw_free[st]));
                            mbar_arrive(smem_u32(&sh.wide_full[w]));
                        }
                        const int i = I.dual ? j >> 1 : j;
                        if (lane == w) {
                            e0 = (I.dual ? !(j & 1) : j < I.n0) ? events0 + I.event(i, 1) : ~0u;
                            e1 = (I.dual ? j & 1 : j < I.n1) ? events1 + I.event(i, 1) : ~0u;
                        }
                        ++tiles;
                    }
                    events0 += I.events(0);
                    events1 += I.events(1);
                }
            }
        }
        __syncwarp();
    } else {
        regs_inc<P::REGS_SOFTMAX>();
        const int t = warp >> 2;
        uint32_t item = 0, events = 0, keys = 0, shares = 0;
        while (true) {
            // The item stays where it is: 128 scores leave few registers.
            bool ok = true;
            if ((warp & 3) == 0) ok = ch_wait(sh, A, sh.item_full[item % CH_ITEMS], item / CH_ITEMS);
            if (group_any(1 + t, !ok)) break;
            const ChunkItem& I = sh.item[item % CH_ITEMS];
            if (I.n0 < 0) break;
            if (!ch_softmax<D, FP8>(sh, A, I, t, events, keys, shares)) break;
            events += I.events(t);
            keys += I.tiles;
            __syncwarp();
            if (lane == 0) free_item(item);
            ++item;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_free(sh.tmem, 512);
    // Every warp has left its waits, so `abort` is final.  Where it is set somebody stopped before all loads had landed: the
    // thread that issued them stays until they have.
    if (tid == 9 * 32 && sh.abort) {
        for (int t = 0; t < 2; ++t)
            if (sh.q_issued[t]) mbar_wait_bounded(smem_u32(&sh.q_full[t]), (sh.q_issued[t] - 1) & 1, A.wait_ns);
        for (int i = max(0, sh.k_issued - P::KS); i < sh.k_issued; ++i)
            mbar_wait_bounded(smem_u32(&sh.k_full[i % P::KS]), (i / P::KS) & 1, A.wait_ns);
        for (int i = max(0, sh.v_issued - P::VS); i < sh.v_issued; ++i)
            mbar_wait_bounded(smem_u32(&sh.v_full[i % P::VS]), (i / P::VS) & 1, A.wait_ns);
        if (sh.tail_open) mbar_wait_bounded(smem_u32(&sh.v_tail), sh.tail_phase & 1, A.wait_ns);
    }
}

// ------------------------------------------------------------------ the join
// Rows of an item that range borders cut: CTA (c, t, x) joins 32 columns x of tile t of the item that begins in range c.
template <int D, bool FP8>
__global__ void __launch_bounds__(CH_ROWS) paged_chunk_join_kernel(const __grid_constant__ ChunkArgs A) {
    __shared__ int slots[CH_CTAS + 1], count;
    grid_wait();
    const int c = blockIdx.x, t = blockIdx.y, row = threadIdx.x;
    const ChunkCut cut = A.cut[c];
    if (cut.last < 0) return;
    const int tl = row / A.r, head = row - tl * A.r, tok = cut.tok0 + t * A.tq + tl;
    const bool real = tl < A.tq && tok < cut.n;
    if (cut.tok0 + t * A.tq >= cut.n) return;
    if (row < 32) {
        int n = 1;
        if (row == 0) slots[0] = 2 * c + 1;
        for (int k0 = c + 1; k0 <= cut.last; k0 += 32) {
            const bool more = k0 + row <= cut.last && A.cut[k0 + row].more;
            const unsigned all = __ballot_sync(0xffffffffu, more);
            if (more) slots[n + __popc(all & ((1u << row) - 1))] = 2 * (k0 + row);
            n += __popc(all);
        }
        if (row == 0) count = n;
    }
    __syncthreads();
    if (!real) return;
    const int n = count;
    float m = -INFINITY, l = 0.f;
    auto part = [&](int i) {       // m, l, c
        const int64_t at = ((int64_t)slots[i] * A.tiles + t) * CH_ROWS + row;
        if (FP8) return reinterpret_cast<const float4*>(A.part_ml)[at];
        const float2 ml = reinterpret_cast<const float2*>(A.part_ml)[at];
        return make_float4(ml.x, ml.y, 0.f, 0.f);
    };
    float cl = 0.f;                // l counts in units of 2^(m - cl)
    bool units = false;
#pragma unroll (FP8 ? 4 : 8)
    for (int i = 0; i < n; ++i) {
        const float4 ml = part(i);
        if (ml.y != 0.f) m = fmaxf(m, ml.x);
        units |= ml.z != 0.f;
    }
    float4 acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
        const int64_t at = (int64_t)slots[i] * A.tiles + t;
        const float4 ml = part(i);
        if (ml.y == 0.f) continue;             // it saw nothing: its memory may hold anything
        const float4* from = reinterpret_cast<const float4*>(A.part_o) + (at * (D / 4) + blockIdx.z * 8) * CH_ROWS + row;
        const float f = ex2(ml.x - m);
        l += f * ml.y;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 o = from[e * CH_ROWS];
            acc[e].x += f * o.x;
            acc[e].y += f * o.y;
            acc[e].z += f * o.z;
            acc[e].w += f * o.w;
        }
    }
    if (FP8 && units) {            // parts whose l counts in units of their own
        ChUnit unit{-INFINITY, 0.f};
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const float4 ml = part(i);
            if (ml.y != 0.f && (unit.m == -INFINITY || ChUnit{ml.x, ml.z}.above(unit))) unit = {ml.x, ml.z};
        }
        unit = unit.with(m);
        l = 0.f;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const float4 ml = part(i);
            if (ml.y != 0.f) l += ChUnit{ml.x, ml.z}.in(unit) * ml.y;
        }
        cl = l != 0.f ? unit.c : 0.f;
    }
    float inv = l != 0.f ? 1.f / l : 0.f;
    if (FP8 && units) {            // (neither 2^c nor 2^c / l need be in fp32's range)
        const float half = truncf(0.5f * cl), a = ex2(half), b = ex2(cl - half);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[e].x = acc[e].x * inv * a * b;
            acc[e].y = acc[e].y * inv * a * b;
            acc[e].z = acc[e].z * inv * a * b;
            acc[e].w = acc[e].w * inv * a * b;
        }
        inv = 1.f;
    }
    const int64_t out = (cut.row + tok) * A.hq + cut.g * A.r + head;
    uint4* to = reinterpret_cast<uint4*>(A.o + out * D + blockIdx.z * 32);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(acc[e].x * inv, acc[e].y * inv), b = __floats2bfloat162_rn(acc[e].z * inv, acc[e].w * inv);
        const __nv_bfloat162 g = __floats2bfloat162_rn(acc[e + 1].x * inv, acc[e + 1].y * inv), d = __floats2bfloat162_rn(acc[e + 1].z * inv, acc[e + 1].w * inv);
        to[e / 2] = make_uint4(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b), *reinterpret_cast<const uint32_t*>(&g),
                               *reinterpret_cast<const uint32_t*>(&d));
    }
    if (blockIdx.z == 0 && A.lse) A.lse[out] = l == 0.f ? -INFINITY : (m - cl + log2f(l) - CH_BIAS_OF<FP8>) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ host
struct ChunkSpace {
    size_t cut, ml, o, q_exp, q8;
    size_t all() const { return cut + ml + o + q_exp + q8; }
};
ChunkSpace chunk_space(int tiles, int d, bool fp8, int64_t q_rows) {
    const size_t rows = (size_t)CH_CTAS * 2 * tiles * CH_ROWS;
    return {round256(CH_CTAS * sizeof(ChunkCut)), round256(rows * (fp8 ? sizeof(float4) : sizeof(float2))), rows * d * sizeof(float), fp8 ? round256((size_t)q_rows) : 0,
            fp8 ? 2 * (size_t)q_rows * d : 0};
}
// Few rows to a request: bound by the bytes of K and V, and products of 128 rows would be mostly empty.
bool chunk_few(int r, int64_t max_new) { return max_new > 0 && max_new <= FEW_ROWS / r; }       // (a product may overflow)
int chunk_tiles(int64_t total_q, int r) { return total_q <= CH_ROWS / r ? 1 : 2; }

const char* chunk_error(const kvo_paged_cache* c, int n_q_heads, int64_t total_q, int64_t max_new, int64_t max_len) {
    if (const char* m = paged_cache_error(c)) return m;
    if (n_q_heads < c->n_kv_heads || n_q_heads % c->n_kv_heads) return "n_q_heads must be a multiple of n_kv_heads";
    if (n_q_heads / c->n_kv_heads > 16) return "n_q_heads / n_kv_heads must be <= 16";
    if (total_q < 0 || total_q > (1 << 30) || total_q * n_q_heads > (1ll << 34)) return "total_q must be in 0..2^30, with at most 2^34 rows of q";
    if (max_new < 0 || max_len < 0) return "max_new and max_len must be >= 0";
    return nullptr;
}

template <int D, bool FP8>
cudaError_t paged_chunk_launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const ChunkArgs& A, cudaStream_t s) {
    using P = ChShape<D, FP8>;
    constexpr int SMEM = P::TILES + (int)sizeof(ChShared);
    static_assert(SMEM <= 227 * 1024 && SMEM > 114 * 1024, "one CTA to an SM");
    static std::atomic<uint64_t> done{0};
    if (first_on_device(done)) {
        const cudaError_t e = cudaFuncSetAttribute(paged_chunk_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        mark_on_device(done);
    }
    const cudaError_t e = launch_dependent(paged_chunk_kernel<D, FP8>, dim3(CH_CTAS), P::THREADS, SMEM, s, 0, mq, mk, mv, A);
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_chunk_join_kernel<D, FP8>, dim3(CH_CTAS, A.tiles, D / 32), CH_ROWS, 0, s, 0, A);
}

}  // namespace kvo

extern "C" kvo_status kvo_paged_chunk_attn_workspace(const kvo_paged_cache* cache, int n_q_heads, int64_t total_q, int64_t max_new,
                                                     int64_t max_len, size_t* bytes_out) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (!bytes_out) return bad("null output pointer");
    *bytes_out = 0;
    if (const char* m = chunk_error(cache, n_q_heads, total_q, max_new, max_len)) return bad(m);
    const int r = n_q_heads / cache->n_kv_heads;
    *bytes_out = chunk_few(r, max_new) ? paged_few_workspace(cache, r, max_new, max_len)
                                       : chunk_space(chunk_tiles(total_q, r), cache->head_dim, cache->format == KVO_PAGES_E4M3, total_q * n_q_heads).all();
    return KVO_OK;
}

extern "C" kvo_status kvo_paged_chunk_attn(const kvo_paged_cache* cache, const void* q, int64_t q_token_stride, int64_t total_q,
                                           int n_q_heads, const int32_t* cu, const int32_t* lens, int64_t max_new, int64_t max_len,
                                           void* o, float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                                           kvo_stream_t stream) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (const char* m = chunk_error(cache, n_q_heads, total_q, max_new, max_len)) return bad(m);
    if (cache->batch == 0 || total_q == 0) return KVO_OK;
    if (!q || !o || !cu || !lens) return bad("null pointer argument");
    if ((uintptr_t)q % 16 || (uintptr_t)o % 16 || (uintptr_t)workspace % 256)
        return bad("q and o must be 16-byte aligned, the workspace 256-byte aligned");
    const int r = n_q_heads / cache->n_kv_heads, D = cache->head_dim;
    const int64_t width = (int64_t)n_q_heads * D, b = cache->batch;
    if (q_token_stride % 8) return bad("strides must be multiples of 8 elements");
    if (q_token_stride < width) return bad("token strides must cover the heads");
    if (q_token_stride > (1ll << 38)) return bad("token strides must be below 2^38 elements");
    const int tiles = chunk_tiles(total_q, r);
    const bool few = chunk_few(r, max_new), fp8 = cache->format == KVO_PAGES_E4M3;
    const ChunkSpace sp = chunk_space(tiles, D, fp8, total_q * n_q_heads);
    const size_t need = few ? paged_few_workspace(cache, r, max_new, max_len) : sp.all();
    if (need && (!workspace || workspace_bytes < need)) return bad("the workspace is too small (kvo_paged_chunk_attn_workspace)");
    const int64_t pool = page_bytes(cache), scales = scale_bytes(cache);
    const Bytes to_o{o, 2 * total_q * width}, to_lse{lse, 4 * total_q * n_q_heads}, to_ws{workspace, (int64_t)need};
    bool meet = meets_any(to_o, {to_lse, to_ws}) || meets_any(to_lse, {to_ws});
    for (const Bytes& x : {to_o, to_lse, to_ws})
        meet |= meets_any(x, {{q, rows_bytes(total_q, q_token_stride, width)}, {cache->k_pages, pool}, {cache->v_pages, pool},
                              {cache->k_scale, scales}, {cache->v_scale, scales}, {cache->table, 4 * b * cache->max_pages}, {lens, 4 * b},
                              {cu, 4 * (b + 1)}});
    if (meet) return bad("o, lse and the workspace must be apart from each other and from all that the call reads");
    const uint64_t rows = (uint64_t)cache->n_pages * cache->n_kv_heads * cache->page_size;
    const int elem = fp8 ? 1 : 2, box = std::min(D * elem, 128), box_rows = few ? 16 : cache->page_size;
    cudaStream_t s = (cudaStream_t)stream;
    CUtensorMap mq, mk, mv;
    if (!tensor_map_rows(&mk, cache->k_pages, elem, D, rows, box, box_rows) || !tensor_map_rows(&mv, cache->v_pages, elem, D, rows, box, box_rows)) {
        set_last_error("cuTensorMapEncodeTiled failed for the pages");
        return KVO_ERR_CUDA;
    }
    if (few) {
        const cudaError_t e = launch_paged_few(cache, mk, mv, q, q_token_stride, total_q, r, cu, lens, max_new, max_len, o, lse, workspace, status, s);
        if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
        return KVO_OK;
    }
    ChunkArgs A{};
    A.k_scale = fp8 ? cache->k_scale : nullptr;
    A.v_scale = fp8 ? cache->v_scale : nullptr;
    A.table = cache->table;
    A.lens = lens;
    A.cu = cu;
    A.o = (uint16_t*)o;
    A.lse = lse;
    A.status = status;
    A.cut = (ChunkCut*)workspace;
    A.part_ml = (uint8_t*)workspace + sp.cut;
    A.part_o = (float*)((uint8_t*)workspace + sp.cut + sp.ml);
    int8_t* const q_exp = (int8_t*)A.part_o + sp.o;
    uint8_t* const q8 = (uint8_t*)q_exp + sp.q_exp;
    A.q_exp = q_exp;
    A.total = total_q;
    A.batch = cache->batch;
    A.hq = n_q_heads;
    A.hkv = cache->n_kv_heads;
    A.r = r;
    A.tq = CH_ROWS / r;
    A.page = cache->page_size;
    A.shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : cache->page_size == 64 ? 6 : 7;
    A.n_pages = cache->n_pages;
    A.max_pages = cache->max_pages;
    A.tiles = tiles;
    // Measured times of 128 keys: one tile of rows is 5/7 of two in bf16 and 4/7 in e4m3 and of d 64; an item in itself costs what
    // 128 keys do.  With 4/7, 5/7 and 6/7, us: 56 single tokens and 8 pieces of 250 behind 512-8192 in bf16 271, 267, 279, in e4m3
    // 269, 292, 318, of d 64 189, 209, 228 and 234, 257, 278; 20 and 4 of 1000 in bf16 615, 613, 615, in e4m3 679, 696, 712.
    A.w1 = fp8 || D == 64 ? 4 : 5;
    A.w2 = 7;
    A.base = 2 * CH_KEYS * A.w2;
    A.least = 2 * CH_KEYS * A.w1 + A.base;
    A.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    A.wide = (uintptr_t)o % 32 == 0;
    A.skip = call_wait.skip;
    A.wait_ns = call_wait.limit_ns;
    const uint64_t sq[3] = {(uint64_t)D, (uint64_t)n_q_heads, (uint64_t)total_q * (fp8 ? 2 : 1)};
    const uint64_t tq[2] = {(uint64_t)D * elem, fp8 ? (uint64_t)width : (uint64_t)q_token_stride * 2};
    const uint32_t bq[3] = {fp8 ? (uint32_t)D : 64u, (uint32_t)r, (uint32_t)A.tq};
    if (!tensor_map(&mq, fp8 ? (const void*)q8 : q, elem, 3, sq, tq, bq)) {
        set_last_error("cuTensorMapEncodeTiled failed for q");
        return KVO_ERR_CUDA;
    }
    if (fp8) {
        const int64_t q_rows = total_q * n_q_heads, ctas = (q_rows * (D / 16) + CS_THREADS - 1) / CS_THREADS;
        const cudaError_t e = launch_dependent(D == 128 ? paged_chunk_split_kernel<128> : paged_chunk_split_kernel<64>, dim3((unsigned)ctas), CS_THREADS, 0, s, 0,
                                               (const uint16_t*)q, q_token_stride, n_q_heads, q_rows, q8, q_exp);
        if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    }
    cudaError_t e;
    if (D == 128) e = fp8 ? paged_chunk_launch<128, true>(mq, mk, mv, A, s) : paged_chunk_launch<128, false>(mq, mk, mv, A, s);
    else e = fp8 ? paged_chunk_launch<64, true>(mq, mk, mv, A, s) : paged_chunk_launch<64, false>(mq, mk, mv, A, s);
    if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    return KVO_OK;
}
