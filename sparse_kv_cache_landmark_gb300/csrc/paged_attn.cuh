// The kernels of kvo_paged_attn, decode attention of one query token per request over a paged cache (bf16, or e4m3 with a
// scale per page and KV head), and, NEW, of kvo_paged_chunk_attn where a request's few new tokens and the query heads of a
// group make at most 16 rows: rows that see different numbers of keys.
//
//   o_h = sum_t softmax_t(q_h . k_t / sqrt(d)) v_t over the tokens of the
//   request (or of the listed blocks of its KV head), lse_h the natural log of
//   the softmax's denominator.
//
// Bound by HBM: each KV head's bytes are read once for all r query heads of its
// group.  Work: the tiles (8 KB of K and V: 32 tokens of 128 e4m3 values) of every
// (request, KV head), laid out group after group, are cut into contiguous ranges
// of equal cost, one per warp, so ragged batches end together; the lengths are
// device data, so each CTA finds its warps' ranges by a prefix sum.  A warp keeps its
// next tiles in flight in its own ring of shared-memory stages, across the borders
// of groups, and waits for no other warp.  TMA fills the stages (128-byte-swizzled
// boxes of 16 rows, so that key and value fragments are read without bank
// conflicts); a page's scales follow by cp.async into the same barrier.  128 KB in
// flight on an SM is enough: with 192 KB 16 x 64K-128K took 450 us instead of 433.
// One pass: running maximum and sum in fp32 registers.
//
// Measured (e4m3, 32 query and 8 KV heads of 128): 16 x 32768 tokens 166 us (6.5 TB/s,
// 0.95 of a measured copy), 16 x 65536-131072 433 us (6.8 TB/s, 1.0), 64 x 256-4096
// 55 us (0.72: about 7 us until the first tile, 5 us for the join), 1 x 131072 56 us.
//
// Tensor cores: mma.sync m16n8k16 on transposed products, S^T = K Q^T and O^T =
// V^T P^T: tokens and value columns are the 16 matrix rows, query heads the 8
// columns, so r <= 8 heads fill one product where heads as rows would leave half
// of it empty.  P^T comes out of S^T by an 8 x 8 transpose in the warp.
// e4m3 codes are widened exactly to f16; q is scaled by a power of two per row, its
// largest value to 2^8..2^9: what is down to 2^-25 of that is exact in f16 as well
// (8 bits above its smallest step, 2^-24), smaller values lose low bits, and below
// 2^-33 they are zero.  The weights exp2(s - m), held times 2^6, are rounded to f16
// next to e4m3 values, whose sum is taken before the rounding (11 bits down to 2^-20
// of the running maximum, steps of 2^-30 of it below), and to bf16 (8 bits) next to
// bf16 values, which have a wider exponent than f16; there o is divided by the sum
// of the rounded weights and lse takes the unrounded one.
// The maximum is only raised when a score passes it by more than 2^8, so most
// tiles have no cross-lane step but one vote.
//
// A group cut by range borders leaves partial (m, l, o) in the workspace, in
// fp32, joined by a second kernel.  Small calls, where latency counts, take one
// cluster per group instead, whose CTAs join through distributed shared memory
// in the same launch: each CTA leaves its part of a row in the memory of the CTA
// that joins it (one barrier; reading the others' parts takes two, and 1 us more).
// Both join in a fixed order: results do not depend on timing.
#pragma once
#include <cuda.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "launch.cuh"
#include "paged.cuh"
#include "tensor_map.cuh"
#include "tma_ptx.cuh"

namespace kvo {

constexpr int PA_WARPS = 4;
constexpr int PA_THREADS = PA_WARPS * 32;
// Tiles that a warp could take in the time it needs to take up a group (64 x 16-8192 tokens: 102 us with 0, 92.4 with 1, 89.4
// with 2, 89.1 with 4; 128 x 500-1000: 46.7, 45.1, 44.9, 46.1).
constexpr int PA_SWITCH = 2;
constexpr int PA_SUB = 16;                    // tokens of a subtile (one k step of the value product, and of a TMA box)
constexpr int PA_RING = 64 * 1024;            // bytes of stages per CTA
// Bytes of the parts that a CTA of a cluster joins: ceil(units / CTAs) slots of as many parts as CTAs, 16 bytes for a lane
// and 16 more each; the most is 8 rows over 6 CTAs (2 x 6 x 528), or 16 rows in runs of 8 lanes over 12 (6 x 12 x 144).
constexpr int pa_parts_bytes(int nh) { return nh == 1 ? 6400 : 10496; }
constexpr float PA_RAISE = 8.f;               // log2: how far a score may pass the running maximum
constexpr float PA_BIAS = 6.f;                // log2: weights are held times 2^6 (f16's small end is 2^-24)

template <int D, bool FP8>
struct PaShape {
    static constexpr int RB = FP8 ? D : 2 * D;               // bytes of a row
    static constexpr int BOX = RB > 128 ? 128 : RB;          // bytes of a box row
    static constexpr int NBOX = RB / BOX;
    static constexpr int SUBS = 256 / RB;                    // subtiles of a tile: 8 KB a stage
    static constexpr int TILE = SUBS * PA_SUB;               // tokens of a tile
    static constexpr int TILE_BYTES = TILE * RB;             // K or V of one tile
    static constexpr int STAGE = 2 * TILE_BYTES;
    static constexpr int STAGES = PA_RING / (PA_WARPS * STAGE);
    static constexpr int KCH = RB / 64;                      // 16-byte chunks of a key row per lane
    static constexpr int STEPS = D / 16;                     // k steps of k . q
    static constexpr int MT = D / 16;                        // m tiles of v^T p
    static constexpr int CHAINS = SUBS > 2 ? 1 : 2;          // accumulators a subtile's scores alternate between
};

struct PagedAttnArgs {
    const uint16_t* q;
    const float* scale[2];
    const int32_t* table;
    const int32_t* lens;
    const int32_t* blocks;        // [G][n_blocks] or NULL: every page of the request
    const int32_t* counts;        // [G] or NULL: n_blocks each
    uint16_t* o;
    float* lse;
    float* part_o;                // [2 warps][r][D]
    float4* part_ml;              // [2 warps][r]: maximum, sum, sum of the rounded weights
    int2* info;                   // [G]: first slot and last warp of a group cut by range borders; x < 0: not cut
    int32_t* status;
    int hkv, r, page, shift, n_pages, max_pages, n_blocks, G;
    int warps;                    // of the range kernel
    float scale_log2;
    long long wait_ns, skip;      // skip: the tile that every warp announces without copying it (tests; -1: none)
    // several new tokens of a request (`NEW`)
    const int32_t* cu;
    int64_t q_stride, total;
    int most;                     // rows of a group at most: room in the workspace, and what the kernel's products hold
};

// The queries of a group are the rows of its products: r heads of one token or, NEW, of each of the request's new tokens.
struct PaRows {
    int64_t first;                // row of q
    int rows, new_tokens;         // rows 0: nothing to serve
};
template <bool NEW>
__device__ __forceinline__ PaRows pa_rows(const PagedAttnArgs& A, int g) {
    if (!NEW) return {g / A.hkv, A.r, 1};
    const int b = g / A.hkv, a = A.cu[b], e = A.cu[b + 1];
    const bool ok = offsets_ascend(a, e, A.total) && (int64_t)(e - a) * A.r <= A.most;
    return {a, ok ? (e - a) * A.r : 0, ok ? e - a : 0};
}
// Where row `row` of group g lies in q (in values) and, as a row of hq heads a token, in o and lse.
template <bool NEW>
__device__ __forceinline__ int64_t pa_out_row(const PagedAttnArgs& A, const PaRows& R, int g, int row) {
    if (!NEW) return (int64_t)g * A.r + row;
    const int token = row / A.r, h = g % A.hkv;
    return (R.first + token) * A.hkv * A.r + h * A.r + row - token * A.r;
}
template <bool NEW>
__device__ __forceinline__ int64_t pa_q_at(const PagedAttnArgs& A, const PaRows& R, int g, int row, int d) {
    if (!NEW) return ((int64_t)g * A.r + row) * d;
    const int token = row / A.r, h = g % A.hkv;
    return (R.first + token) * A.q_stride + (int64_t)(h * A.r + row - token * A.r) * d;
}

__device__ __forceinline__ int pa_len(const PagedAttnArgs& A, int b) {
    return min(max(A.lens[b], 0), A.max_pages * A.page);
}
// Tokens of group g that its tiles cover: the request's, or whole listed blocks.
template <bool NEW>
__device__ __forceinline__ int pa_span(const PagedAttnArgs& A, int g) {
    if (NEW) return pa_rows<NEW>(A, g).rows ? pa_len(A, g / A.hkv) : 0;
    if (A.blocks) return (A.counts ? min(max(A.counts[g], 0), A.n_blocks) : A.n_blocks) * A.page;
    return pa_len(A, g / A.hkv);
}

// A length or count out of range is clamped, a request with bad offsets or too many rows left out; say so.
template <bool NEW>
__device__ __forceinline__ void pa_check_counts(const PagedAttnArgs& A, int g) {
    if (!A.status) return;
    if (NEW && pa_rows<NEW>(A, g).rows == 0 && A.cu[g / A.hkv] != A.cu[g / A.hkv + 1]) atomicOr(A.status, KVO_DEV_BAD_COUNT);
    const int len = A.lens[g / A.hkv];
    const bool bad_count = !NEW && A.counts && (A.counts[g] < 0 || A.counts[g] > A.n_blocks);
    if (len < 0 || len > (int64_t)A.max_pages * A.page || bad_count) atomicOr(A.status, KVO_DEV_BAD_COUNT);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool FP8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (FP8)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// The same for weights, no larger than f16's largest value: where fp32's steps are 8 or more (scores from 2^26 on) the roundings of
// the rise that is let pass and of the bias may make one 2^16.
__device__ __forceinline__ uint32_t pack_weights_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Transposes an 8 x 8 block of 16-bit values over the warp (lane (g, c): row g, columns 2c, 2c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// One warp's running state; lane (g, c) = (lane / 4, lane % 4).  The products are computed transposed, tokens
// (or value columns) as the 16 matrix rows and query heads as columns, 8 to a block: r <= 8 fills one block
// where heads as rows would leave half of every product empty.  The lane holds heads 8 x + 2c, 8 x + 2c + 1.
template <int D, bool FP8, int NH>
struct PaState {
    float o[PaShape<D, FP8>::MT][NH][4];   // [..][x][2 i + e]: value column pa_col(2 j + i, g), head 8 x + 2c + e
    float m[NH][2], l[NH][2];              // l: this lane's share of the sum
    float lw[NH][2];                       // the sum of the rounded weights (bf16 only)
    float vs;                              // the value scale that o is held in
};

// Scores and values of one tile; nv[s] of subtile s's 16 tokens are real, and (NEW) the lane's rows see the first see[..] of
// the tile's (FULL: all of them).
template <int D, bool FP8, int NH, bool FULL, bool NEW>
__device__ __forceinline__ void pa_tile(PaState<D, FP8, NH>& T, const uint32_t (&qf)[PaShape<D, FP8>::STEPS][NH][2],
                                        const float (&qs)[NH][2], const uint8_t* ksm, const uint8_t* vsm,
                                        const float (&kscale)[PaShape<D, FP8>::SUBS],
                                        const float (&vscale)[PaShape<D, FP8>::SUBS],
                                        const int (&nv)[PaShape<D, FP8>::SUBS], const int (&see)[NH][2]) {
    using S = PaShape<D, FP8>;
    constexpr int BOXROWS = S::TILE * 128;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float sc[S::SUBS][NH][S::CHAINS][4];
#pragma unroll
    for (int u = 0; u < S::SUBS; ++u)
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int k = 0; k < S::CHAINS; ++k) sc[u][x][k][e] = 0.f;
#pragma unroll
    for (int m = 0; m < S::KCH; ++m)
#pragma unroll
        for (int u = 0; u < S::SUBS; ++u) {
            uint32_t w[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 16 * u + 8 * i + g;
                const uint8_t* a;
                if (S::BOX == 128) a = ksm + (m >> 1) * BOXROWS + row * 128 + (((2 * c + (m & 1)) ^ (row & 7)) << 4);
                else a = ksm + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
                const uint4 v = *reinterpret_cast<const uint4*>(a);
                w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
            }
            constexpr int PER = FP8 ? 4 : 2;                 // k steps of a chunk
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                uint32_t a[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    a[i] = FP8 ? e4m3x2_to_f16x2((uint16_t)w[i][s]) : w[i][(2 * s) & 3];
                    a[i + 2] = FP8 ? e4m3x2_to_f16x2((uint16_t)(w[i][s] >> 16)) : w[i][(2 * s + 1) & 3];
                }
#pragma unroll
                for (int x = 0; x < NH; ++x)
                    mma16816<FP8>(sc[u][x][s & (S::CHAINS - 1)], a, qf[PER * m + s][x][0], qf[PER * m + s][x][1]);
            }
        }
    float mx[NH][2];
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mx[x][e] = -INFINITY;
#pragma unroll
            for (int u = 0; u < S::SUBS; ++u) {
                const float f = qs[x][e] * kscale[u];
                constexpr int L = S::CHAINS - 1;
                sc[u][x][0][e] = (L ? sc[u][x][0][e] + sc[u][x][L][e] : sc[u][x][0][e]) * f;
                sc[u][x][0][e + 2] = (L ? sc[u][x][0][e + 2] + sc[u][x][L][e + 2] : sc[u][x][0][e + 2]) * f;
                if (!FULL) {
                    if (g >= nv[u]) sc[u][x][0][e] = -INFINITY;
                    if (g + 8 >= nv[u]) sc[u][x][0][e + 2] = -INFINITY;
                    if (NEW && 16 * u + g >= see[x][e]) sc[u][x][0][e] = -INFINITY;
                    if (NEW && 16 * u + g + 8 >= see[x][e]) sc[u][x][0][e + 2] = -INFINITY;
                }
                mx[x][e] = fmaxf(mx[x][e], fmaxf(sc[u][x][0][e], sc[u][x][0][e + 2]));
            }
        }
    bool raise = false;
#pragma unroll
    for (int x = 0; x < NH; ++x) raise |= mx[x][0] > T.m[x][0] + PA_RAISE || mx[x][1] > T.m[x][1] + PA_RAISE;
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) mx[x][e] = fmaxf(mx[x][e], __shfl_xor_sync(0xffffffffu, mx[x][e], o));
                const float m = fmaxf(T.m[x][e], mx[x][e]);
                const float f = T.m[x][e] == -INFINITY ? 0.f : ex2(T.m[x][e] - m);
                T.m[x][e] = m;
                T.l[x][e] *= f;
                if (!FP8) T.lw[x][e] *= f;
#pragma unroll
                for (int j = 0; j < S::MT; ++j) { T.o[j][x][e] *= f; T.o[j][x][e + 2] *= f; }
            }
    }
    float fold[S::SUBS];           // what a weight is multiplied by so that o stays in units of T.vs
    if (FP8) {
        float top = vscale[0];
#pragma unroll
        for (int u = 1; u < S::SUBS; ++u) top = fmaxf(top, vscale[u]);
        if (top > T.vs) {          // uniform over the warp
            const float f = T.vs / top;
            T.vs = top;
#pragma unroll
            for (int j = 0; j < S::MT; ++j)
#pragma unroll
                for (int x = 0; x < NH; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) T.o[j][x][e] *= f;
        }
#pragma unroll
        for (int u = 0; u < S::SUBS; ++u) fold[u] = vscale[u] == T.vs ? 1.f : vscale[u] / T.vs;
    }
    uint32_t pb[S::SUBS][NH][2];   // the weights as the right operand: rows are tokens
#pragma unroll
    for (int u = 0; u < S::SUBS; ++u)
#pragma unroll
        for (int x = 0; x < NH; ++x) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float m = T.m[x][e & 1];
                p[e] = ex2(sc[u][x][0][e] + (PA_BIAS - (m == -INFINITY ? 0.f : m)));
                T.l[x][e & 1] += p[e];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t v = FP8 ? pack_weights_f16(p[2 * i] * fold[u], p[2 * i + 1] * fold[u]) : pack_bf(p[2 * i], p[2 * i + 1]);
                if (!FP8) {
                    // o is divided by the sum of the weights as the product takes them: a bf16 rounding (2^-8)
                    // shared by numerator and denominator cancels where few tokens carry the weight
                    T.lw[x][0] += bf16lo_to_f32(v);
                    T.lw[x][1] += bf16hi_to_f32(v);
                }
                pb[u][x][i] = transpose8(v);
            }
        }
    // values: this lane's token rows 2c, 2c + 1, 2c + 8, 2c + 9 of each subtile
    constexpr int VW = S::RB == 64 ? 2 : 4;                  // 32-bit words of a chunk (8 bytes: d 64 in e4m3)
    constexpr int MC = FP8 ? 2 : 1;                          // m tiles (pairs of columns) a word holds
#pragma unroll
    for (int b = 0; b < S::NBOX; ++b)
#pragma unroll
        for (int u = 0; u < S::SUBS; ++u) {
            uint32_t w[4][VW];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int tr = 16 * u + 2 * c + (k & 1) + 8 * (k >> 1);
                if (S::BOX == 128) {
                    const uint4 v = *reinterpret_cast<const uint4*>(vsm + b * BOXROWS + tr * 128 + ((g ^ (tr & 7)) << 4));
                    w[k][0] = v.x; w[k][1] = v.y; w[k][VW - 2] = v.z; w[k][VW - 1] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(vsm + tr * 64 + ((((g >> 1) ^ ((tr >> 1) & 3)) << 4) | ((g & 1) << 3)));
                    w[k][0] = v.x; w[k][1] = v.y;
                }
                if (!FULL && tr - 16 * u >= nv[u])            // what lies behind the end may be NaN: 0 * NaN must not reach o
#pragma unroll
                    for (int i = 0; i < VW; ++i) w[k][i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                // per column of the word: the tokens 2c, 2c + 1 and 2c + 8, 2c + 9 as pairs
                if (FP8) {
                    const uint32_t x0 = __byte_perm(w[0][i], w[1][i], 0x5140), x1 = __byte_perm(w[2][i], w[3][i], 0x5140);
                    const uint32_t y0 = __byte_perm(w[0][i], w[1][i], 0x7362), y1 = __byte_perm(w[2][i], w[3][i], 0x7362);
                    const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)x0), e4m3x2_to_f16x2((uint16_t)(x0 >> 16)),
                                           e4m3x2_to_f16x2((uint16_t)x1), e4m3x2_to_f16x2((uint16_t)(x1 >> 16))};
                    const uint32_t d[4] = {e4m3x2_to_f16x2((uint16_t)y0), e4m3x2_to_f16x2((uint16_t)(y0 >> 16)),
                                           e4m3x2_to_f16x2((uint16_t)y1), e4m3x2_to_f16x2((uint16_t)(y1 >> 16))};
                    const int j = (b * VW + i) * MC;
#pragma unroll
                    for (int x = 0; x < NH; ++x) {
                        mma16816<FP8>(T.o[j][x], a, pb[u][x][0], pb[u][x][1]);
                        mma16816<FP8>(T.o[j + MC - 1][x], d, pb[u][x][0], pb[u][x][1]);
                    }
                } else {
                    const uint32_t a[4] = {__byte_perm(w[0][i], w[1][i], 0x5410), __byte_perm(w[0][i], w[1][i], 0x7632),
                                           __byte_perm(w[2][i], w[3][i], 0x5410), __byte_perm(w[2][i], w[3][i], 0x7632)};
                    const int j = (b * VW + i) * MC;
#pragma unroll
                    for (int x = 0; x < NH; ++x) mma16816<FP8>(T.o[j][x], a, pb[u][x][0], pb[u][x][1]);
                }
            }
        }
}

// Value column that lane row g holds in place q of the order of pa_tile (accumulator j covers places 2 j, 2 j + 1).
template <int D, bool FP8>
__device__ __forceinline__ int pa_col(int q, int g) {
    if (FP8) return g * (D / 8) + q;
    return (q >> 3) * 64 + g * 8 + (q & 7);
}

// What one lane knows of a page of its group: its entry of the table, which is not looked at before the page is
// needed (so that the load of a batch ahead holds nobody up), and its real tokens (0: nothing to read).
struct PaPage {
    int entry, tokens;
};

template <bool NEW>
__device__ __forceinline__ PaPage pa_page(const PagedAttnArgs& A, int g, int i) {
    PaPage P{0, 0};
    if (g >= A.G || i >= (pa_span<NEW>(A, g) + A.page - 1) >> A.shift) return P;
    const int b = g / A.hkv;
    int logical = i;
    if (!NEW && A.blocks) {
        logical = __ldg(A.blocks + (int64_t)g * A.n_blocks + i);
        if (logical < 0 || logical >= A.max_pages) {
            if (A.status) atomicOr(A.status, KVO_DEV_BAD_BLOCK_ID);
            return P;
        }
    }
    P.tokens = max(min(A.page, pa_len(A, b) - logical * A.page), 0);
    if (P.tokens > 0) P.entry = __ldg(A.table + (int64_t)b * A.max_pages + logical);
    return P;
}

// Kept beside a stage: the group of the tile in it and that group's tiles, its first token, and its subtiles' scales and real
// tokens.
template <int SUBS>
struct PaInfo {
    float ks[SUBS], vs[SUBS];
    int nv[SUBS], g, n, tok;
};

// Copies 4 bytes to shared memory; mbar gets the thread's arrival once its copies before have landed.
__device__ __forceinline__ void copy4(void* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_copied(uint32_t mbar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(mbar) : "memory");
}
__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// Whole warp: the queries of group g on their way.
template <int D, bool NEW>
__device__ __forceinline__ void pa_prefetch(const PagedAttnArgs& A, int g) {
    const int lane = threadIdx.x & 31;
    if (NEW) {
        const PaRows R = pa_rows<NEW>(A, g);
        for (int i = lane * 64; i < R.rows * D; i += 32 * 64) prefetch_l1(A.q + pa_q_at<NEW>(A, R, g, i / D, D) + i % D);
    } else {
        for (int i = lane * 64; i < A.r * D; i += 32 * 64) prefetch_l1(A.q + (int64_t)g * A.r * D + i);
    }
}
// Query fragments of group g: heads 8 x + lane / 4 as columns (heads beyond r: zero), and the scores' factors of the
// lane's heads 8 x + 2c, 8 x + 2c + 1.
template <int D, bool FP8, int NH, bool NEW>
__device__ __forceinline__ void pa_query(const PagedAttnArgs& A, const PaRows& R, int g, uint32_t (&qf)[PaShape<D, FP8>::STEPS][NH][2],
                                         float (&qs)[NH][2]) {
    using S = PaShape<D, FP8>;
    const int lane = threadIdx.x & 31, gr = lane >> 2, c = lane & 3;
#pragma unroll
    for (int x = 0; x < NH; ++x) {
        const int head = gr + 8 * x;
        const uint16_t* q = A.q + (head < R.rows ? pa_q_at<NEW>(A, R, g, head, D) : 0);
        float amax = 0.f;
#pragma unroll
        for (int m = 0; m < S::KCH; ++m) {
            constexpr int ES = FP8 ? 1 : 2, PER = FP8 ? 4 : 2;
            const int box = S::BOX == 128 ? m >> 1 : 0, ch = S::BOX == 128 ? 2 * c + (m & 1) : c;
            const int e0 = box * (128 / ES) + ch * (16 / ES);
#pragma unroll
            for (int s = 0; s < PER; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t v = head < R.rows ? *reinterpret_cast<const uint32_t*>(q + e0 + 4 * s + 2 * k) : 0u;
                    qf[PER * m + s][x][k] = v;
                    amax = fmaxf(amax, fmaxf(fabsf(bf16lo_to_f32(v)), fabsf(bf16hi_to_f32(v))));
                }
        }
        float scale = A.scale_log2;
        if (FP8) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // row / 2^(e - 8): the largest value is in [2^8, 2^9)
            const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -110), 126);
            const float f = __uint_as_float((uint32_t)(8 - e + 127) << 23);
            scale = A.scale_log2 * __uint_as_float((uint32_t)(e - 8 + 127) << 23);
#pragma unroll
            for (int s = 0; s < S::STEPS; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t v = qf[s][x][k];
                    qf[s][x][k] = pack_f16(bf16lo_to_f32(v) * f, bf16hi_to_f32(v) * f);
                }
        }
        // head 8 x + h's scale sits in lanes 4 h ..
        qs[x][0] = __shfl_sync(0xffffffffu, scale, 8 * c);
        qs[x][1] = __shfl_sync(0xffffffffu, scale, 8 * c + 4);
    }
}

// After a wait that ran out: the status bit, and what came too late gets as long again.  Of `stages` stages bit i of
// `phase` is the parity that stage i's next fill would have.
static __device__ __noinline__ void pa_late(uint32_t bar, int stages, uint32_t phase, long long limit, int32_t* status) {
    if ((threadIdx.x & 31) == 0 && status) atomicOr(status, KVO_DEV_TIMEOUT);
    for (int i = 0; i < stages; ++i) mbar_wait_bounded(bar + 8 * i, ((phase >> i) & 1) ^ 1, limit);
    __syncwarp();
}

// One warp attends to `count` tiles in a row, from tile t0 of group g0 on and, unless ONE, through the groups after it.
// The copies run STAGES tiles ahead, across groups.  finish(T, g, its tiles, first, count) takes each group's state.
// Returns whether every wait was met; every copy issued has landed in any case.
template <int D, bool FP8, int NH, bool ONE, bool NEW, typename F>
__device__ __forceinline__ bool pa_run(const PagedAttnArgs& A, const CUtensorMap* map_k, const CUtensorMap* map_v,
                                       uint32_t ring, const uint8_t* ring_p, uint32_t bar,
                                       PaInfo<PaShape<D, FP8>::SUBS>* info, int g0, int t0, long long count, F&& finish) {
    using S = PaShape<D, FP8>;
    const int lane = threadIdx.x & 31;
    // Pages come in batches of 32, one per lane; the next batch, of this group or of the one after, is fetched while
    // this one is used.
    int bg = g0, base = (t0 * S::TILE) >> A.shift, ng = bg, nbase = base;
    auto next_batch = [&]() {
        nbase += 32;
        if ((nbase << A.shift) < pa_span<NEW>(A, ng)) return pa_page<NEW>(A, ng, nbase + lane);
        if constexpr (ONE) {
            return PaPage{0, 0};
        } else {
            do ++ng; while (ng < A.G && pa_span<NEW>(A, ng) <= 0);
            nbase = 0;
            return pa_page<NEW>(A, ng, lane);
        }
    };
    int page, tokens;              // of this lane's page of the batch in use; -1: the table's entry is out of range
    auto use = [&](const PaPage& P) {
        const bool bad = P.tokens > 0 && (P.entry < 0 || P.entry >= A.n_pages);
        page = bad ? -1 : P.entry;
        tokens = bad ? 0 : P.tokens;
        if (bad && A.status) atomicOr(A.status, KVO_DEV_BAD_BLOCK_ID);
    };
    use(pa_page<NEW>(A, bg, base + lane));
    PaPage nxt{0, 0};
    bool fetched = false;          // nxt is the batch at (ng, nbase)
    // the next tile to issue: its group, that group's KV head and tiles
    int ig = g0, ih = g0 % A.hkv, it = t0, in = (pa_span<NEW>(A, g0) + S::TILE - 1) / S::TILE;
    int st_in = 0;
    long long issued = 0;
    auto issue = [&]() {
        if (!ONE && it >= in) {
            do in = (pa_span<NEW>(A, ++ig) + S::TILE - 1) / S::TILE; while (in <= 0);   // the count ends before the groups do
            it = 0;
            ih = ig % A.hkv;
            pa_prefetch<D, NEW>(A, ig);        // its queries are wanted in a moment
        }
        const int tok = it * S::TILE, pg = tok >> A.shift;
        if (ig != bg || pg - base >= 32) {
            if (!fetched) nxt = next_batch();
            bg = ng;
            base = nbase;
            use(nxt);
            nxt = next_batch();
            fetched = true;
        }
        // lane u takes subtile u
        const int mine = tok + (lane & (S::SUBS - 1)) * PA_SUB, my_pg = mine >> A.shift, k = (my_pg - base) & 31;
        const int off = mine - (my_pg << A.shift);
        const int my_page = __shfl_sync(0xffffffffu, page, k);
        const int nv = min(max(__shfl_sync(0xffffffffu, tokens, k) - off, 0), PA_SUB);
        const uint32_t b = bar + 8 * st_in, dst = ring + st_in * S::STAGE;
        const uint32_t have = __ballot_sync(0xffffffffu, lane < S::SUBS && nv > 0);
        if (lane < S::SUBS) info[st_in].nv[lane] = nv;
        if (lane == 0) {
            info[st_in].g = ig;
            info[st_in].n = in;
            if (NEW) info[st_in].tok = tok;
            if (have) mbar_expect_tx(b, __popc(have) * (S::STAGE / S::SUBS));
        }
        __syncwarp();
        if ((have >> lane & 1) && issued != A.skip) {
            const int slot = my_page * A.hkv + ih, row = slot * A.page + off;
#pragma unroll
            for (int x = 0; x < S::NBOX; ++x) {
                const uint32_t at = dst + x * (S::TILE * 128) + lane * (PA_SUB * S::BOX);
                tma_load_2d(at, map_k, x * (128 / (FP8 ? 1 : 2)), row, b);
                tma_load_2d(at + S::TILE_BYTES, map_v, x * (128 / (FP8 ? 1 : 2)), row, b);
            }
            if (FP8) {
                copy4(&info[st_in].ks[lane], A.scale[0] + slot);
                copy4(&info[st_in].vs[lane], A.scale[1] + slot);
            }
        } else if (lane < S::SUBS) {
            info[st_in].ks[lane] = info[st_in].vs[lane] = 0.f;
        }
        if (FP8 && have && lane < S::SUBS) arrive_copied(b);
        if (++st_in == S::STAGES) st_in = 0;
        ++it;
        ++issued;
    };
    while (issued < min(count, (long long)S::STAGES)) issue();
    if (!fetched) {
        nxt = next_batch();
        fetched = true;
    }

    uint32_t qf[S::STEPS][NH][2];
    float qs[NH][2];
    PaState<D, FP8, NH> T;
    int see[NH][2], see_all = 0;   // NEW: tokens of the request that the lane's rows see, and that all rows do
    PaRows R{0, A.r, 1};
    auto begin = [&](int g) {
        if (NEW) {
            R = pa_rows<NEW>(A, g);
            const int past = pa_len(A, g / A.hkv) - R.new_tokens;
            see_all = past + 1;
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) see[x][e] = past + 1 + (8 * x + 2 * (lane & 3) + e) / A.r;
        }
        pa_query<D, FP8, NH, NEW>(A, R, g, qf, qs);
#pragma unroll
        for (int x = 0; x < NH; ++x) {
#pragma unroll
            for (int j = 0; j < S::MT; ++j) T.o[j][x][0] = T.o[j][x][1] = T.o[j][x][2] = T.o[j][x][3] = 0.f;
            T.m[x][0] = T.m[x][1] = -INFINITY;
            T.l[x][0] = T.l[x][1] = T.lw[x][0] = T.lw[x][1] = 0.f;
        }
        T.vs = 0.f;
    };
    int cg = g0, cn = 0, first = t0, done = 0, st = 0;
    uint32_t phase = 0;            // bit i: parity of stage i's next wait
    bool dead = false;
    begin(cg);
    // Every copy issued is waited for, also after a wait that ran out: none may land once the CTA has left.
    for (long long c = 0; c < issued; ++c) {
        const PaInfo<S::SUBS>& I = info[st];
        if (!ONE && I.g != cg) {
            finish(T, cg, cn, first, done);
            cg = I.g;
            first = done = 0;
            begin(cg);
        }
        cn = I.n;
        int nv[S::SUBS];
        bool some = false, all = true;
#pragma unroll
        for (int u = 0; u < S::SUBS; ++u) {
            nv[u] = I.nv[u];
            some |= nv[u] > 0;
            all &= nv[u] == PA_SUB;
        }
        int here[NH][2];
        if (NEW) {
            all &= I.tok + S::TILE <= see_all;
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) here[x][e] = see[x][e] - I.tok;
        }
        if (some) {
            if (!mbar_wait_bounded(bar + 8 * st, (phase >> st) & 1, A.wait_ns)) dead = true;
            phase ^= 1u << st;
            float ks[S::SUBS], vs[S::SUBS];
#pragma unroll
            for (int u = 0; u < S::SUBS; ++u) {
                ks[u] = FP8 ? I.ks[u] : 1.f;
                vs[u] = FP8 ? I.vs[u] : 1.f;
            }
            const uint8_t* tile = ring_p + st * S::STAGE;
            if (dead) {
            } else if (all) {
                pa_tile<D, FP8, NH, true, NEW>(T, qf, qs, tile, tile + S::TILE_BYTES, ks, vs, nv, here);
            } else {
                pa_tile<D, FP8, NH, false, NEW>(T, qf, qs, tile, tile + S::TILE_BYTES, ks, vs, nv, here);
            }
        }
        if (++st == S::STAGES) st = 0;
        ++done;
        dead = __any_sync(0xffffffffu, dead);
        if (issued < count && !dead) issue();
    }
    if (dead) pa_late(bar, S::STAGES, phase, A.wait_ns, A.status);
    finish(T, cg, cn, first, done);
    return !dead;
}

// The sums of a state over the warp's token lanes.
template <int D, bool FP8, int NH>
__device__ __forceinline__ void pa_sum(const PaState<D, FP8, NH>& T, int x, int e, float& l, float& lw) {
    l = T.l[x][e];
    lw = FP8 ? 0.f : T.lw[x][e];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        if (!FP8) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    }
    if (FP8) lw = l;
}

// The shared memory of both kernels: stages, what is kept beside them, and their barriers.
template <int D, bool FP8>
struct PaShared {
    uint64_t bars[PA_WARPS][PaShape<D, FP8>::STAGES];
    PaInfo<PaShape<D, FP8>::SUBS> info[PA_WARPS][PaShape<D, FP8>::STAGES];
};
template <int D, bool FP8>
__device__ __forceinline__ void pa_init(PaShared<D, FP8>& sh) {
    const int warp = threadIdx.x >> 5;
    // a stage is full with its tiles and, in e4m3, each subtile's scales
    if ((threadIdx.x & 31) == 0)
        for (int i = 0; i < PaShape<D, FP8>::STAGES; ++i)
            mbar_init(smem_u32(&sh.bars[warp][i]), FP8 ? 1 + PaShape<D, FP8>::SUBS : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
}

// NEW, whole warp: whether no earlier request with good offsets ends behind the first row of group g's request (`sorted`:
// no offset is below the one before it, so none can).
__device__ __forceinline__ bool pa_alone(const PagedAttnArgs& A, int g, bool sorted) {
    if (sorted) return true;
    const int b = g / A.hkv, a = A.cu[b];
    bool ok = true;
    for (int i = threadIdx.x & 31; i < b; i += 32) ok &= !(offsets_ascend(A.cu[i], A.cu[i + 1], A.total) && A.cu[i + 1] > a);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && A.status) atomicOr(A.status, KVO_DEV_BAD_COUNT);
    return ok;
}

// 64-bit divisions are long; most numbers here are short.
__device__ __forceinline__ long long pa_div(long long a, long long b) {
    return (a | b) >> 31 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// One thread-block cluster per group: its warps split the group's tiles, and the states are joined through shared
// memory, then through distributed shared memory.
template <int D, bool FP8, int NH, bool NEW>
__global__ void __launch_bounds__(PA_THREADS, NH == 1 ? 3 : 2)
paged_cluster_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ PagedAttnArgs A) {
    using S = PaShape<D, FP8>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PaShared<D, FP8> sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* ring_p = smem_raw + (ring - smem_u32(smem_raw));
    // After the copies the ring's memory holds the warps' states, [4][r][D + 4]; behind it is what the cluster's CTAs leave
    // to this one to join.
    float* mrg = reinterpret_cast<float*>(ring_p);
    float* parts = reinterpret_cast<float*>(ring_p + PA_RING);
    constexpr int MS = D + 4;
    cluster_arrive();              // this CTA has started: others may write to its memory
    pa_init(sh);
    if (tid == 0) { tensor_map_prefetch(&map_k); tensor_map_prefetch(&map_v); }
    grid_wait();
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int g = blockIdx.x / size, n = (pa_span<NEW>(A, g) + S::TILE - 1) / S::TILE;
    if (tid == 0 && rank == 0) pa_check_counts<NEW>(A, g);
    const PaRows R = pa_rows<NEW>(A, g);
    bool sorted = true;
    if (NEW)
        for (int i = tid; i < g / A.hkv; i += PA_THREADS) sorted &= A.cu[i] <= A.cu[i + 1];
    const int warps = PA_WARPS * size, me = rank * PA_WARPS + warp;
    const int t0 = (int)pa_div((long long)n * me, warps), t1 = (int)pa_div((long long)n * (me + 1), warps);
    pa_prefetch<D, NEW>(A, g);
    const int ws = warp * S::STAGES * S::STAGE;
    pa_run<D, FP8, NH, true, NEW>(A, &map_k, &map_v, ring + ws, ring_p + ws, smem_u32(sh.bars[warp]), sh.info[warp], g, t0, t1 - t0,
                             [&](PaState<D, FP8, NH>& T, int, int, int, int) {
        if (NEW) sorted = __syncthreads_and(sorted);
        else __syncthreads();      // the ring is free
        const int gr = lane >> 2, c = lane & 3;
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l, lw;
                pa_sum(T, x, e, l, lw);
                const int head = 8 * x + 2 * c + e;
                if (head < R.rows) {
                    float* dst = mrg + (warp * R.rows + head) * MS;
                    if (gr == 0) { dst[D] = T.m[x][e]; dst[D + 1] = l; dst[D + 2] = lw; dst[D + 3] = FP8 ? T.vs : 1.f; }
#pragma unroll
                    for (int j = 0; j < S::MT; ++j) {
                        dst[pa_col<D, FP8>(2 * j, gr)] = T.o[j][x][e];
                        dst[pa_col<D, FP8>(2 * j + 1, gr)] = T.o[j][x][e + 2];
                    }
                }
            }
    });
    __syncthreads();
    cluster_wait();                // all have started
    const bool alone = !NEW || pa_alone(A, g, sorted);
    // A row is cut into runs of W lanes with 4 columns each, which are joined by the CTAs in turn: unit u (row and run) by CTA
    // u % size, as its slot u / size.  Every CTA leaves its part of a unit, its columns and (maximum, sum, sum of the rounded
    // weights), in the joining CTA's memory.  There a warp's 32 / W groups of lanes take every (32 / W)-th part, and lane k of
    // 16 part k's maximum and sums.
    auto join = [&](auto width) {
        constexpr int W = decltype(width)::value, N = 32 / W, RUNS = D / (4 * W), MOST = 16;    // CTAs of a cluster at most
        constexpr int STRIDE = 4 * W + 4;                           // floats of a part
        for (int i = tid; i < R.rows * (D / 4); i += PA_THREADS) {
            const int row = i / (D / 4), col = (i - row * (D / 4)) * 4;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < PA_WARPS; ++w) m = fmaxf(m, mrg[(w * R.rows + row) * MS + D]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f, lw = 0.f;
#pragma unroll
            for (int w = 0; w < PA_WARPS; ++w) {
                const float* src = mrg + (w * R.rows + row) * MS;
                const float4 ml = *reinterpret_cast<const float4*>(src + D), o = *reinterpret_cast<const float4*>(src + col);
                if (ml.y == 0.f) continue;
                const float f = ex2(ml.x - m), fo = f * ml.w;
                l += f * ml.y;
                lw += f * ml.z;
                acc.x += fo * o.x;
                acc.y += fo * o.y;
                acc.z += fo * o.z;
                acc.w += fo * o.w;
            }
            const int u = row * RUNS + col / (4 * W), slot = u / (int)size, to = u - slot * (int)size;
            float* dst = parts + (slot * size + rank) * STRIDE;
            st_cluster_f32x4(dst + col % (4 * W), to, acc);
            if (col % (4 * W) == 0) st_cluster_f32x4(dst + 4 * W, to, make_float4(m, l, lw, 0.f));
        }
        cluster_barrier();
        for (int slot = warp; slot * (int)size + (int)rank < R.rows * RUNS; slot += PA_WARPS) {
            const int u = slot * size + rank, row = u / RUNS, col = ((u - row * RUNS) * W + lane % W) * 4;
            const float* src = parts + slot * size * STRIDE;
            float4 ml = make_float4(-INFINITY, 0.f, 0.f, 0.f), acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane % MOST < size) ml = *reinterpret_cast<const float4*>(src + (lane % MOST) * STRIDE + 4 * W);
            float m = ml.x;
#pragma unroll
            for (int i = 1; i < MOST; i <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
            const float f = ml.y == 0.f ? 0.f : ex2(ml.x - m);
            float l = f * ml.y, lw = f * ml.z;
#pragma unroll
            for (int i = 1; i < MOST; i <<= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, i);
                if (!FP8) lw += __shfl_xor_sync(0xffffffffu, lw, i);
            }
            if (FP8) lw = l;
#pragma unroll
            for (int i = 0; i < MOST / N; ++i) {
                const int k = N * i + lane / W;
                const float c = __shfl_sync(0xffffffffu, f, k, MOST);
                if (k < size) {
                    const float4 o = *reinterpret_cast<const float4*>(src + k * STRIDE + (lane % W) * 4);
                    acc.x += c * o.x; acc.y += c * o.y; acc.z += c * o.z; acc.w += c * o.w;
                }
            }
#pragma unroll
            for (int i = W; i < 32; i <<= 1) {
                acc.x += __shfl_xor_sync(0xffffffffu, acc.x, i);
                acc.y += __shfl_xor_sync(0xffffffffu, acc.y, i);
                acc.z += __shfl_xor_sync(0xffffffffu, acc.z, i);
                acc.w += __shfl_xor_sync(0xffffffffu, acc.w, i);
            }
            const int64_t to = pa_out_row<NEW>(A, R, g, row);
            const bool some = lw != 0.f;
            if (NEW && !alone) continue;
            if (lane < W)
                *reinterpret_cast<uint2*>(A.o + to * D + col) =
                    make_uint2(some ? pack_bf(acc.x / lw, acc.y / lw) : 0u, some ? pack_bf(acc.z / lw, acc.w / lw) : 0u);
            if (lane < W && col == 0 && (!NEW || A.lse)) A.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l) - PA_BIAS) * 0.6931471805599453f;
        }
    };
    // Large clusters have more warps than rows: they take runs of 32 columns (before the parts were left to the joining CTA,
    // 1 x 4096, 16 CTAs: 10.3 us, 10.9 with whole rows; but 32 x 512, one CTA: 13.8, and 12.5 with whole rows).
    if (size > 8) join(std::integral_constant<int, 8>());
    else join(std::integral_constant<int, D / 4>());
}

// Ranges of all groups' tiles, of equal cost, one per warp.
template <int D, bool FP8, int NH, bool NEW>
__global__ void __launch_bounds__(PA_THREADS, 2)
paged_range_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ PagedAttnArgs A) {
    using S = PaShape<D, FP8>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PaShared<D, FP8> sh;
    __shared__ long long s_scan[2][PA_WARPS], s_to[2][PA_THREADS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint8_t* ring_p = smem_raw + (ring - smem_u32(smem_raw));
    auto tiles_of = [&](int g) { return (pa_span<NEW>(A, g) + S::TILE - 1) / S::TILE; };
    pa_init(sh);
    if (tid == 0) { tensor_map_prefetch(&map_k); tensor_map_prefetch(&map_v); }
    grid_wait();
    // Ranges are equal in cost: a group's tiles and PA_SWITCH for taking it up.  Prefixes of both over the CTA, by
    // requests, or by groups where each has a list of its own: each thread's share, then shuffles within a warp, then the
    // warps' totals through shared memory.
    const int heads = !NEW && A.blocks ? 1 : A.hkv, stride = NEW ? A.most : A.r;
    bool sorted = true;
    const int units = A.G / heads, per = (units + PA_THREADS - 1) / PA_THREADS;
    auto cost_of = [](int n) { return n > 0 ? n + PA_SWITCH : 0; };
    long long cost = 0, tiles = 0, total = 0;
    for (int i = 0; i < per; ++i) {
        const int u = tid * per + i;
        if (u >= units) break;
        const int n = tiles_of(u * heads);
        tiles += (long long)heads * n;
        cost += (long long)heads * cost_of(n);
        if (blockIdx.x == 0) pa_check_counts<NEW>(A, u * heads);
        if (NEW) sorted &= A.cu[u] <= A.cu[u + 1];
    }
    long long cost_to = cost, tiles_to = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, cost_to, o), y = __shfl_up_sync(0xffffffffu, tiles_to, o);
        if (lane >= o) { cost_to += x; tiles_to += y; }
    }
    if (lane == 31) { s_scan[0][warp] = cost_to; s_scan[1][warp] = tiles_to; }
    if (NEW) sorted = __syncthreads_and(sorted);
    else __syncthreads();
    long long all_tiles = 0;
#pragma unroll
    for (int w = 0; w < PA_WARPS; ++w) {
        if (w < warp) { cost_to += s_scan[0][w]; tiles_to += s_scan[1][w]; }
        total += s_scan[0][w];
        all_tiles += s_scan[1][w];
    }
    s_to[0][tid] = cost_to - cost;
    s_to[1][tid] = tiles_to - tiles;
    __syncthreads();
    grid_launch_next();            // the join's CTAs may take their places; they wait for this grid's end
    // a cost of two at least to a warp, at most 512 parts to join for a group, and warps spread over the CTAs before they
    // fill them
    const long long n_warp = max(1ll, min(min((long long)gridDim.x * PA_WARPS, 512ll * A.G), total / 2));
    const long long each = pa_div(total, n_warp), extra = total - each * n_warp;    // the first `extra` warps take one more
    auto start = [&](long long w) { return w < n_warp ? each * w + min(w, extra) : total; };
    // The border at cost x, by the warp: the group it falls in, that group's cost prefix, and the tile it lies before, x less
    // the prefix and PA_SWITCH, or the first.  Returns that tile's number among all.
    auto border = [&](long long x, int& g, int& in, long long& before) {
        if (x >= total) return all_tiles;
        int seg = -1;
#pragma unroll
        for (int i = 0; i < PA_THREADS; i += 32) seg += __popc(__ballot_sync(0xffffffffu, s_to[0][i + lane] <= x));
        long long c = s_to[0][seg], t = s_to[1][seg];
        for (int u = seg * per;; ++u) {
            const int n = u < units ? tiles_of(u * heads) : 0, k = cost_of(n);
            if (u == seg * per + per - 1 || x < c + (long long)k * heads) {
                const int h = (int)pa_div(x - c, max(k, 1));
                before = c + (long long)h * k;
                g = u * heads + h;
                in = max((int)(x - before) - PA_SWITCH, 0);
                return t + (long long)h * n + in;
            }
            c += (long long)k * heads;
            t += (long long)n * heads;
        }
    };
    const long long me = (long long)warp * gridDim.x + blockIdx.x;
    int g0 = 0, t0 = 0, g1, t1;
    long long before = 0, before1;     // cost of the groups before the one being finished
    const long long at = border(start(me), g0, t0, before), count = border(start(me + 1), g1, t1, before1) - at;
    // groups with nothing to attend to
    for (int g = blockIdx.x; g < A.G; g += gridDim.x)
        if (tiles_of(g) == 0) {
            if (NEW) {
                const PaRows R = pa_rows<NEW>(A, g);
                const bool alone = pa_alone(A, g, sorted);
                for (int i = tid; alone && i < R.rows * D; i += PA_THREADS) A.o[pa_out_row<NEW>(A, R, g, i / D) * D + i % D] = 0;
                for (int i = tid; alone && A.lse && i < R.rows; i += PA_THREADS) A.lse[pa_out_row<NEW>(A, R, g, i)] = -INFINITY;
            } else {
                for (int i = tid; i < A.r * D; i += PA_THREADS) A.o[(int64_t)g * A.r * D + i] = 0;
                for (int i = tid; i < A.r; i += PA_THREADS) A.lse[(int64_t)g * A.r + i] = -INFINITY;
            }
            if (tid == 0) A.info[g] = make_int2(-1, -1);
        }
    if (count <= 0) return;
    int seg = 0;
    const int ws = warp * S::STAGES * S::STAGE;
    pa_run<D, FP8, NH, false, NEW>(A, &map_k, &map_v, ring + ws, ring_p + ws, smem_u32(sh.bars[warp]), sh.info[warp], g0, t0, count, [&](PaState<D, FP8, NH>& T, int g, int n, int first, int done) {
        const bool whole = done == n;
        const long long slot = 2 * me + (seg ? 1 : 0);
        const int gr = lane >> 2, c = lane & 3;
        const PaRows R = pa_rows<NEW>(A, g);
        const bool alone = !NEW || pa_alone(A, g, sorted);
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l, lw;
                pa_sum(T, x, e, l, lw);
                const int head = 8 * x + 2 * c + e;
                if (head >= R.rows || (NEW && !alone)) continue;
                const float m = T.m[x][e];
                const int64_t row = whole ? pa_out_row<NEW>(A, R, g, head) : slot * stride + head;
                // the lane's columns are runs of 8 places of the order of pa_tile
                const float f = whole ? (lw != 0.f ? (FP8 ? T.vs : 1.f) / lw : 0.f) : FP8 ? T.vs : 1.f;
#pragma unroll
                for (int q = 0; q < 2 * S::MT; q += 8) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) { v[2 * i] = T.o[q / 2 + i][x][e] * f; v[2 * i + 1] = T.o[q / 2 + i][x][e + 2] * f; }
                    const int64_t at = row * D + pa_col<D, FP8>(q, gr);
                    if (whole) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = lw != 0.f ? pack_bf(v[2 * i], v[2 * i + 1]) : 0u;
                        *reinterpret_cast<uint4*>(A.o + at) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        *reinterpret_cast<float4*>(A.part_o + at) = make_float4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<float4*>(A.part_o + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
                if (gr == 0) {
                    if (whole) { if (!NEW || A.lse) A.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l) - PA_BIAS) * 0.6931471805599453f; }
                    else A.part_ml[row] = make_float4(m, l, lw, 0.f);
                }
            }
        if (lane == 0 && (whole || !alone)) A.info[g] = make_int2(-1, -1);
        else if (lane == 0 && first == 0) {
            // the warp that holds the group's last tile
            const long long last = before + PA_SWITCH + n - 1, wide = extra * (each + 1);
            const long long w = last < wide ? last / (each + 1) : extra + (last - wide) / each;
            A.info[g] = make_int2((int)slot, (int)w);
        }
        before += n + PA_SWITCH;
        ++seg;
    });
}

// Joins the parts of groups cut by range borders.  `slices` warps (1, 2, 4 or 8) take a (group, head): warp s adds
// parts s, s + slices, .. of 4 or 2 value columns a lane, and the slices are added in order.
constexpr int PA_JOIN = 8;         // warps of a CTA
template <int D, bool NEW>
__global__ void __launch_bounds__(PA_JOIN * 32) paged_join_kernel(const __grid_constant__ PagedAttnArgs A, int slices) {
    constexpr int N = D / 32;
    __shared__ float s_acc[PA_JOIN][D], s_m[PA_JOIN], s_l[PA_JOIN][2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = warp % slices;
    const int64_t pair = ((int64_t)blockIdx.x * PA_JOIN + warp) / slices;
    grid_wait();
    const int rows = NEW ? A.most : A.r;
    const bool in = pair < (int64_t)A.G * rows;
    const int g = in ? (int)(pair / rows) : 0, row = in ? (int)(pair - (int64_t)g * rows) : 0;
    const PaRows R = pa_rows<NEW>(A, g);
    const bool have = in && row < R.rows;
    const int2 info = A.info[g];
    // A warp whose wait ran out leaves the words of the groups after it as they were in the workspace, whatever that is:
    // only a range of this launch's warps is read, so that nothing past the workspace is, and no more parts than warps.
    const bool cut = have && info.x >= 0 && info.x / 2 <= info.y && info.y < A.warps;
    const int n = cut ? info.y - info.x / 2 + 1 : 0;          // parts: the first warp's slot, then slot 0 of each warp after it
    auto part = [&](int i) { return (i == 0 ? (int64_t)info.x : 2 * ((int64_t)(info.x / 2) + i)) * rows + row; };
    auto values = [&](int i, float (&o)[N]) {
        const float* at = A.part_o + part(i) * D + N * lane;
        if constexpr (N == 4) {
            const float4 v = *reinterpret_cast<const float4*>(at);
            o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(at);
            o[0] = v.x; o[1] = v.y;
        }
    };
    // the first parts' values are on their way while the maxima are compared
    constexpr int AHEAD = 4;
    float o0[AHEAD][N];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (slice + k * slices < n) values(slice + k * slices, o0[k]);
    float m = -INFINITY;
    for (int i = slice * 32 + lane; i < n; i += slices * 32) m = fmaxf(m, A.part_ml[part(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (slices > 1) {
        if (lane == 0) s_m[warp] = m;
        __syncthreads();
        for (int i = 0; i < slices; ++i) m = fmaxf(m, s_m[warp - slice + i]);
    }
    float acc[N], l = 0.f, lw = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    auto add = [&](int i, const float (&o)[N]) {
        const float4 ml = A.part_ml[part(i)];
        const float f = ex2(ml.x - m);
        if (ml.y != 0.f) {         // an empty part adds nothing, whatever its maximum
            l += f * ml.y;
            lw += f * ml.z;
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += f * o[e];
        }
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (slice + k * slices < n) add(slice + k * slices, o0[k]);
#pragma unroll 8
    for (int i = slice + AHEAD * slices; i < n; i += slices) {
        float o[N];
        values(i, o);
        add(i, o);
    }
    if (slices > 1) {
#pragma unroll
        for (int e = 0; e < N; ++e) s_acc[warp][N * lane + e] = acc[e];
        if (lane == 0) { s_l[warp][0] = l; s_l[warp][1] = lw; }
        __syncthreads();
        if (slice) return;
        for (int i = 1; i < slices; ++i) {
            l += s_l[warp + i][0];
            lw += s_l[warp + i][1];
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += s_acc[warp + i][N * lane + e];
        }
    }
    if (!cut) return;
    const int64_t to = pa_out_row<NEW>(A, R, g, row);
#pragma unroll
    for (int e = 0; e < N; e += 2)
        *reinterpret_cast<uint32_t*>(A.o + to * D + N * lane + e) = lw != 0.f ? pack_bf(acc[e] / lw, acc[e + 1] / lw) : 0u;
    if (lane == 0 && (!NEW || A.lse)) A.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l) - PA_BIAS) * 0.6931471805599453f;
}

struct PaPlan {
    int cluster, ctas;
};
constexpr int PA_SLOTS = 2 * 152;             // CTAs of the range kernel
PaPlan paged_attn_plan(int64_t groups, int r, int64_t max_tokens);
size_t round256(size_t x);
size_t paged_attn_workspace(const PaPlan& plan, int G, int r, int d);

template <int D, bool FP8, int NH, bool NEW>
inline cudaError_t paged_attn_launch(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttnArgs& A, const PaPlan& plan,
                                     cudaStream_t s) {
    const int smem = PA_RING + 1024, smem_cluster = smem + pa_parts_bytes(NH);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = cudaSuccess;
    if (first_on_device(done)) {
        e = cudaFuncSetAttribute(paged_cluster_kernel<D, FP8, NH, NEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_cluster);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(paged_cluster_kernel<D, FP8, NH, NEW>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(paged_range_kernel<D, FP8, NH, NEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        mark_on_device(done);
    }
    if (plan.cluster)
        return launch_dependent(paged_cluster_kernel<D, FP8, NH, NEW>, plan.ctas, PA_THREADS, smem_cluster, s, plan.cluster, mk, mv, A);
    e = launch_dependent(paged_range_kernel<D, FP8, NH, NEW>, plan.ctas, PA_THREADS, smem, s, 0, mk, mv, A);
    if (e != cudaSuccess) return e;
    // as many warps to a pair as keep them in one wave: 5 CTAs of 8 to an SM (50 registers a thread)
    const int64_t pairs = (int64_t)A.G * (NEW ? A.most : A.r);
    int slices = PA_JOIN;
    while (slices > 1 && pairs * slices > 152 * 40) slices /= 2;
    const dim3 grid((unsigned)((pairs * slices + PA_JOIN - 1) / PA_JOIN));
    return launch_dependent(paged_join_kernel<D, NEW>, grid, PA_JOIN * 32, 0, s, 0, A, slices);
}

}  // namespace kvo
