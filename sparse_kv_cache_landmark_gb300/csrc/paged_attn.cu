// kvo_paged_attn: decode attention of one query token per request over a paged
// cache (bf16, or e4m3 with a scale per page and KV head).
//
//   o_h = sum_t softmax_t(q_h . k_t / sqrt(d)) v_t over the tokens of the
//   request (or of the listed blocks of its KV head), lse_h the natural log of
//   the softmax's denominator.
//
// Bound by HBM: each KV head's bytes are read once for all r query heads of
// its group.  Work: the 32-token tiles of every (request, KV head), laid out
// group after group, are cut into equal contiguous ranges, one per CTA (the
// lengths are device data, so each CTA finds its own range by a prefix sum);
// ragged batches therefore end together.  Within a range a group's tiles are
// split over the CTA's four warps; each warp keeps its next tiles in flight in
// its own ring of shared-memory stages, filled by TMA (128-byte-swizzled boxes
// of 16 rows, so that both the key and the value fragments are read without
// bank conflicts).  One pass: running maximum and sum in fp32 registers.
//
// Tensor cores: mma.sync m16n8k16 on transposed products, S^T = K Q^T and O^T =
// V^T P^T: tokens and value columns are the 16 matrix rows, query heads the 8
// columns, so r <= 8 heads fill one product where heads as rows would leave half
// of it empty (435 -> about 250 instructions per 16 tokens).  P^T comes out of S^T by
// an 8 x 8 transpose in the warp.  e4m3 codes are widened exactly to f16; q is
// scaled by a power of two per row so that it is exact in f16 as well down to
// 2^-32 of its row's largest value.  The weights exp2(s - m) are rounded to f16
// (11 bits) next to e4m3 values, whose sum is taken before the rounding, and to
// bf16 (8 bits) next to bf16 values, which have a wider exponent than f16; there o
// is divided by the sum of the rounded weights and lse takes the unrounded one.
// The maximum is only raised when a score passes it by more than 2^8, so most
// tiles have no cross-lane step but one vote.
//
// A group cut by range borders leaves partial (m, l, o) in the workspace, in
// fp32, joined by a second kernel.  Small calls, where latency counts, take one
// cluster per group instead, whose CTAs join through distributed shared memory
// in the same launch.  Both join in a fixed order: results do not depend on timing.
#include <cuda.h>
#include <stdio.h>

#include <algorithm>

#include "launch.cuh"
#include "paged.cuh"
#include "tensor_map.cuh"
#include "tma_ptx.cuh"

namespace kvo {

constexpr int PA_WARPS = 4;
constexpr int PA_THREADS = PA_WARPS * 32;
constexpr int PA_SUB = 16;                    // tokens of a subtile (one k step of the value product, and of a TMA box)
constexpr int PA_RING = 96 * 1024;            // bytes of stages per CTA
constexpr int PA_PER_SM = 2;                  // CTAs per SM: 96 KB of stages each
constexpr float PA_RAISE = 8.f;               // log2: how far a score may pass the running maximum
constexpr float PA_BIAS = 6.f;                // log2: weights are held times 2^6 (f16's small end is 2^-24)

template <int D, bool FP8>
struct PaShape {
    static constexpr int RB = FP8 ? D : 2 * D;               // bytes of a row
    static constexpr int BOX = RB > 128 ? 128 : RB;          // bytes of a box row
    static constexpr int NBOX = RB / BOX;
    static constexpr int SUBS = RB > 128 ? 1 : 2;            // subtiles of a tile (8 KB a stage at most)
    static constexpr int TILE = SUBS * PA_SUB;               // tokens of a tile
    static constexpr int TILE_BYTES = TILE * RB;             // K or V of one tile
    static constexpr int STAGE = 2 * TILE_BYTES;
    static constexpr int STAGES = PA_RING / (PA_WARPS * STAGE);
    static constexpr int KCH = RB / 64;                      // 16-byte chunks of a key row per lane
    static constexpr int STEPS = D / 16;                     // k steps of k . q
    static constexpr int MT = D / 16;                        // m tiles of v^T p
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
    float* part_o;                // [2 ctas][r][D]
    float4* part_ml;              // [2 ctas][r]: maximum, sum, sum of the rounded weights
    int2* info;                   // [G]: first and last CTA of a group cut by range borders; x < 0: not cut
    int32_t* status;
    int batch, hkv, r, page, shift, n_pages, max_pages, n_blocks, G;
    float scale_log2;
    long long wait_ns;
};

__device__ __forceinline__ int pa_len(const PagedAttnArgs& A, int b) {
    return min(max(A.lens[b], 0), A.max_pages * A.page);
}
// Tokens of group g that its tiles cover: the request's, or whole listed blocks.
__device__ __forceinline__ int pa_span(const PagedAttnArgs& A, int g) {
    if (A.blocks) return (A.counts ? min(max(A.counts[g], 0), A.n_blocks) : A.n_blocks) * A.page;
    return pa_len(A, g / A.hkv);
}

// A length or count out of range is clamped; say so.
__device__ __forceinline__ void pa_check_counts(const PagedAttnArgs& A, int g) {
    if (!A.status) return;
    const int len = A.lens[g / A.hkv];
    const bool bad_count = A.counts && (A.counts[g] < 0 || A.counts[g] > A.n_blocks);
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

// Scores and values of one tile; nv[s] of subtile s's 16 tokens are real (all: nv_all).
template <int D, bool FP8, int NH>
__device__ __forceinline__ void pa_tile(PaState<D, FP8, NH>& T, const uint32_t (&qf)[PaShape<D, FP8>::STEPS][NH][2],
                                        const float (&qs)[NH][2], const uint8_t* ksm, const uint8_t* vsm,
                                        const float (&kscale)[PaShape<D, FP8>::SUBS],
                                        const float (&vscale)[PaShape<D, FP8>::SUBS],
                                        const int (&nv)[PaShape<D, FP8>::SUBS], bool all) {
    using S = PaShape<D, FP8>;
    constexpr int BOXROWS = S::TILE * 128;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float sc[S::SUBS][NH][2][4];                             // two chains each, so that products follow closer
#pragma unroll
    for (int u = 0; u < S::SUBS; ++u)
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[u][x][0][e] = sc[u][x][1][e] = 0.f;
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
                    mma16816<FP8>(sc[u][x][s & 1], a, qf[PER * m + s][x][0], qf[PER * m + s][x][1]);
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
                sc[u][x][0][e] = (sc[u][x][0][e] + sc[u][x][1][e]) * f;
                sc[u][x][0][e + 2] = (sc[u][x][0][e + 2] + sc[u][x][1][e + 2]) * f;
                if (!all) {
                    if (g >= nv[u]) sc[u][x][0][e] = -INFINITY;
                    if (g + 8 >= nv[u]) sc[u][x][0][e + 2] = -INFINITY;
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
        if (S::SUBS > 1) top = fmaxf(top, vscale[S::SUBS - 1]);
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
                const uint32_t v = FP8 ? pack_f16(p[2 * i] * fold[u], p[2 * i + 1] * fold[u]) : pack_bf(p[2 * i], p[2 * i + 1]);
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
                if (!all && tr - 16 * u >= nv[u])            // what lies behind the end may be NaN: 0 * NaN must not reach o
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

// What one lane knows of a batch of 32 pages of the segment: page, scales, tokens.
struct PaPage {
    int row;          // first row of the page in the pool seen as [n_pages * Hkv * page] rows; < 0: skip
    int tokens;       // real tokens of the page
    float ks, vs;
};

__device__ __forceinline__ PaPage pa_page(const PagedAttnArgs& A, int g, int i, int len, int n_logical) {
    PaPage P{-1, 0, 0.f, 0.f};
    if (i >= n_logical) return P;
    const int b = g / A.hkv, h = g - b * A.hkv;
    int logical = i;
    if (A.blocks) {
        logical = __ldg(A.blocks + (int64_t)g * A.n_blocks + i);
        if (logical < 0 || logical >= A.max_pages) {
            if (A.status) atomicOr(A.status, KVO_DEV_BAD_BLOCK_ID);
            return P;
        }
    }
    P.tokens = min(A.page, len - logical * A.page);
    if (P.tokens <= 0) return P;
    const int page = __ldg(A.table + (int64_t)b * A.max_pages + logical);
    if (page < 0 || page >= A.n_pages) {
        if (A.status) atomicOr(A.status, KVO_DEV_BAD_BLOCK_ID);
        P.tokens = 0;
        return P;
    }
    P.row = (page * A.hkv + h) * A.page;
    if (A.scale[0]) {
        P.ks = __ldg(A.scale[0] + (int64_t)page * A.hkv + h);
        P.vs = __ldg(A.scale[1] + (int64_t)page * A.hkv + h);
    } else {
        P.ks = P.vs = 1.f;
    }
    return P;
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void pa_store(const PagedAttnArgs& A, int64_t row, int d, int col, float acc, float m, float l,
                                         float lw) {
    A.o[row * d + col] = __bfloat16_as_ushort(__float2bfloat16_rn(lw != 0.f ? acc / lw : 0.f));
    if (col == 0) A.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l) - PA_BIAS) * 0.6931471805599453f;
}

// CLU: one thread-block cluster per group splits the group's tiles and joins its CTAs' states through distributed
// shared memory.  Else: equal ranges of all groups' tiles, parts joined by the second kernel.
template <int D, bool FP8, int NH, bool CLU>
__global__ void __launch_bounds__(PA_THREADS, PA_PER_SM)
paged_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ PagedAttnArgs A) {
    using S = PaShape<D, FP8>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[PA_WARPS * S::STAGES];
    __shared__ long long s_pre, s_scan[PA_WARPS];
    __shared__ int s_g, s_dead;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* ring_p = smem_raw + (ring - smem_u32(smem_raw));
    // Outside a segment's copies the ring's memory also holds the warps' states, [4][r][D + 4], and the CTA's, [r][D + 4].
    float* mrg = reinterpret_cast<float*>(ring_p);
    float* cl = reinterpret_cast<float*>(ring_p + 48 * 1024);
    constexpr int MS = D + 4;
    const uint32_t wring = ring + warp * S::STAGES * S::STAGE;
    const uint8_t* wring_p = ring_p + warp * S::STAGES * S::STAGE;
    const uint32_t wbar = smem_u32(bars) + warp * S::STAGES * 8;
    if (lane == 0)
        for (int i = 0; i < S::STAGES; ++i) mbar_init(wbar + 8 * i, 1);
    if (tid == 0) s_dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    auto tiles_of = [&](int g) { return (pa_span(A, g) + S::TILE - 1) / S::TILE; };

    grid_wait();
    long long total = 0, n_cta = 1, lo = 0, hi = 0, gpre = 0;
    int g = 0;
    if constexpr (CLU) {
        const uint32_t rank = cluster_rank(), size = cluster_size();
        g = blockIdx.x / size;
        const int n = tiles_of(g);
        lo = (long long)n * rank / size;
        hi = (long long)n * (rank + 1) / size;
        if (tid == 0 && rank == 0) pa_check_counts(A, g);
        __syncthreads();
    } else {
    // this CTA's range of the tiles of all groups
    const int per = (A.G + PA_THREADS - 1) / PA_THREADS;
    long long sum = 0;
    for (int i = 0; i < per; ++i) {
        const int g = tid * per + i;
        if (g >= A.G) break;
        sum += tiles_of(g);
        if (blockIdx.x == 0) pa_check_counts(A, g);
    }
    // inclusive prefix over the CTA: shuffles within a warp, the warps' totals through shared memory
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < PA_WARPS; ++w) {
        if (w < warp) inc += s_scan[w];
        total += s_scan[w];
    }
    const long long pre = inc - sum;
    n_cta = max(1ll, min((long long)gridDim.x, total));                      // a tile for each, so every range holds work
    lo = blockIdx.x < n_cta ? total * blockIdx.x / n_cta : total;
    hi = blockIdx.x < n_cta ? total * (blockIdx.x + 1) / n_cta : total;
    if (lo >= pre && lo < pre + sum) {
        long long at = pre;
        for (int i = 0; i < per; ++i) {
            const int k = tid * per + i;
            const int n = k < A.G ? tiles_of(k) : 0;
            if (lo < at + n) { s_g = k; s_pre = at; break; }
            at += n;
        }
    }
    __syncthreads();
    // groups with nothing to attend to
    for (int k = blockIdx.x; k < A.G; k += gridDim.x)
        if (tiles_of(k) == 0) {
            for (int i = tid; i < A.r * D; i += PA_THREADS) A.o[(int64_t)k * A.r * D + i] = 0;
            for (int i = tid; i < A.r; i += PA_THREADS) A.lse[(int64_t)k * A.r + i] = -INFINITY;
            if (tid == 0) A.info[k] = make_int2(-1, -1);
        }
    grid_launch_next();            // the join's CTAs may take their places; they wait for this grid's end
    if (lo >= hi) return;
    g = s_g;
    gpre = s_pre;
    }

    uint32_t phase = 0;            // bit i: parity of stage i's next wait
    long long cur = lo;
    int seg = 0;
    bool dead = false;
    while (CLU || cur < hi) {      // a cluster's CTA has one segment, empty or not
        const int n = tiles_of(g);
        if (!CLU && cur >= gpre + n) { gpre += n; ++g; continue; }
        const int t0 = (int)(cur - gpre), t1 = CLU ? (int)hi : (int)min((long long)n, hi - gpre);
        const int len = pa_len(A, g / A.hkv);
        const int n_logical = (pa_span(A, g) + A.page - 1) >> A.shift;
        // this warp's tiles
        const int w0 = t0 + (int)((long long)(t1 - t0) * warp / PA_WARPS);
        const int w1 = t0 + (int)((long long)(t1 - t0) * (warp + 1) / PA_WARPS);

        // tiles w0..w1: pages come in batches of 32, one per lane; the next batch is loaded while this one is used
        int base = (w0 * S::TILE) >> A.shift;
        PaPage cur_p = pa_page(A, g, base + lane, len, n_logical), nxt_p = pa_page(A, g, base + 32 + lane, len, n_logical);
        int issued = w0;
        // first row in the pool of the subtile at token t of the span, and its real tokens (up to a batch ahead)
        auto find = [&](int t, int& row, int& tok) {
            const int pg = t >> A.shift, k = pg - base, off = t - (pg << A.shift);
            row = __shfl_sync(0xffffffffu, k < 32 ? cur_p.row : nxt_p.row, k & 31) + off;
            tok = __shfl_sync(0xffffffffu, k < 32 ? cur_p.tokens : nxt_p.tokens, k & 31) - off;
        };
        const bool wide = A.page >= S::TILE;                 // a tile lies within one page
        int st_in = 0, st_out = 0; // stages of the next tile to issue and to use
        auto issue = [&](int t) {  // copies of tile t into its stage: each subtile that has tokens
            const uint32_t bar = wbar + 8 * st_in, dst = wring + st_in * S::STAGE;
            if (++st_in == S::STAGES) st_in = 0;
            int row[S::SUBS], tok[S::SUBS];
            find(t * S::TILE, row[0], tok[0]);
            if (S::SUBS > 1) {
                row[S::SUBS - 1] = row[0] + PA_SUB;
                tok[S::SUBS - 1] = tok[0] - PA_SUB;
                if (!wide) find(t * S::TILE + PA_SUB, row[S::SUBS - 1], tok[S::SUBS - 1]);
            }
            if (lane == 0) {
                int n_sub = 0;
#pragma unroll
                for (int u = 0; u < S::SUBS; ++u) n_sub += tok[u] > 0;
                if (n_sub) mbar_expect_tx(bar, n_sub * (S::STAGE / S::SUBS));
#pragma unroll
                for (int u = 0; u < S::SUBS; ++u)
                    if (tok[u] > 0) {
#pragma unroll
                        for (int x = 0; x < S::NBOX; ++x) {
                            const uint32_t at = dst + x * (S::TILE * 128) + u * (PA_SUB * S::BOX);
                            tma_load_2d(at, &map_k, x * (128 / (FP8 ? 1 : 2)), row[u], bar);
                            tma_load_2d(at + S::TILE_BYTES, &map_v, x * (128 / (FP8 ? 1 : 2)), row[u], bar);
                        }
                    }
            }
        };
        for (; issued < min(w1, w0 + S::STAGES);) issue(issued++);

        // query fragments: heads 8 x + lane / 4 of the group as columns (heads beyond r: zero)
        uint32_t qf[S::STEPS][NH][2];
        float qs[NH][2];
        {
            const int gr = lane >> 2, c = lane & 3;
            const uint16_t* qg = A.q + (int64_t)g * A.r * D;
#pragma unroll
            for (int x = 0; x < NH; ++x) {
                const int head = gr + 8 * x;
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
                            const uint32_t v = head < A.r ? *reinterpret_cast<const uint32_t*>(qg + head * D + e0 + 4 * s + 2 * k) : 0u;
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
                // head 8 x + h's scale sits in lanes 4 h ..: this lane needs heads 2c and 2c + 1
                qs[x][0] = __shfl_sync(0xffffffffu, scale, 8 * c);
                qs[x][1] = __shfl_sync(0xffffffffu, scale, 8 * c + 4);
            }
        }
        PaState<D, FP8, NH> T;
#pragma unroll
        for (int x = 0; x < NH; ++x) {
#pragma unroll
            for (int j = 0; j < S::MT; ++j) T.o[j][x][0] = T.o[j][x][1] = T.o[j][x][2] = T.o[j][x][3] = 0.f;
            T.m[x][0] = T.m[x][1] = -INFINITY;
            T.l[x][0] = T.l[x][1] = T.lw[x][0] = T.lw[x][1] = 0.f;
        }
        T.vs = 0.f;

        // Every copy issued is waited for, also after a wait that ran out: none may land once the CTA has left.
        for (int t = w0; t < issued; ++t) {
            const int pg = (t * S::TILE) >> A.shift;
            if (pg - base >= 32) {
                base += 32;
                cur_p = nxt_p;
                nxt_p = pa_page(A, g, base + 32 + lane, len, n_logical);
            }
            float ks[S::SUBS], vs[S::SUBS];
            int nv[S::SUBS];
            const int k = pg - base, off = t * S::TILE - (pg << A.shift);
            const int tok = __shfl_sync(0xffffffffu, cur_p.tokens, k) - off;
            nv[0] = min(PA_SUB, tok);
            ks[0] = __shfl_sync(0xffffffffu, cur_p.ks, k);
            vs[0] = __shfl_sync(0xffffffffu, cur_p.vs, k);
            if (S::SUBS > 1) {
                constexpr int U = S::SUBS - 1;
                nv[U] = min(PA_SUB, tok - PA_SUB);
                ks[U] = ks[0];
                vs[U] = vs[0];
                if (!wide) {       // pages of 16 tokens: the next page, of the same batch (tiles start at even pages)
                    nv[U] = __shfl_sync(0xffffffffu, cur_p.tokens, (k + 1) & 31);
                    ks[U] = __shfl_sync(0xffffffffu, cur_p.ks, (k + 1) & 31);
                    vs[U] = __shfl_sync(0xffffffffu, cur_p.vs, (k + 1) & 31);
                }
            }
            const bool some = nv[0] > 0 || nv[S::SUBS - 1] > 0, all = nv[0] == PA_SUB && nv[S::SUBS - 1] == PA_SUB;
            const int st = st_out;
            if (++st_out == S::STAGES) st_out = 0;
            if (some) {
                if (!mbar_wait_bounded(wbar + 8 * st, (phase >> st) & 1, A.wait_ns)) dead = true;
                phase ^= 1u << st;
                if (!dead)
                    pa_tile<D, FP8, NH>(T, qf, qs, wring_p + st * S::STAGE, wring_p + st * S::STAGE + S::TILE_BYTES, ks, vs, nv, all);
            }
            dead = __any_sync(0xffffffffu, dead);
            if (issued < w1 && !dead) issue(issued++);
        }
        if (dead && lane == 0) {   // a copy never came: say so, and leave once every thread knows
            if (A.status) atomicOr(A.status, KVO_DEV_TIMEOUT);
            s_dead = 1;
        }
        __syncthreads();           // the ring is free
        if (!CLU && s_dead) return;
        // the warps' states
        {
            const int gr = lane >> 2, c = lane & 3;
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float l = T.l[x][e], lw = FP8 ? l : T.lw[x][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        l += __shfl_xor_sync(0xffffffffu, l, o);
                        if (!FP8) lw += __shfl_xor_sync(0xffffffffu, lw, o);
                    }
                    if (FP8) lw = l;
                    const int head = 8 * x + 2 * c + e;
                    if (head < A.r) {
                        float* dst = mrg + (warp * A.r + head) * MS;
                        if (gr == 0) { dst[D] = T.m[x][e]; dst[D + 1] = l; dst[D + 2] = lw; dst[D + 3] = FP8 ? T.vs : 1.f; }
#pragma unroll
                        for (int j = 0; j < S::MT; ++j) {
                            dst[pa_col<D, FP8>(2 * j, gr)] = T.o[j][x][e];
                            dst[pa_col<D, FP8>(2 * j + 1, gr)] = T.o[j][x][e + 2];
                        }
                    }
                }
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == n;
        const int slot = 2 * blockIdx.x + (seg ? 1 : 0);
        for (int i = tid; i < A.r * D; i += PA_THREADS) {
            const int row = i / D, col = i - row * D;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < PA_WARPS; ++w) m = fmaxf(m, mrg[(w * A.r + row) * MS + D]);
            float acc = 0.f, l = 0.f, lw = 0.f;
#pragma unroll
            for (int w = 0; w < PA_WARPS; ++w) {
                const float* src = mrg + (w * A.r + row) * MS;
                if (src[D + 1] == 0.f) continue;
                const float f = ex2(src[D] - m);
                l += f * src[D + 1];
                lw += f * src[D + 2];
                acc += f * src[D + 3] * src[col];
            }
            if constexpr (CLU) {
                float* dst = cl + row * MS;
                dst[col] = acc;
                if (col == 0) { dst[D] = m; dst[D + 1] = l; dst[D + 2] = lw; }
            } else if (whole) {
                pa_store(A, (int64_t)g * A.r + row, D, col, acc, m, l, lw);
            } else {
                const int64_t at = (int64_t)slot * A.r + row;
                A.part_o[at * D + col] = acc;
                if (col == 0) A.part_ml[at] = make_float4(m, l, lw, 0.f);
            }
        }
        if constexpr (CLU) {
            cluster_barrier();
            const uint32_t rank = cluster_rank(), size = cluster_size();
            for (int i = tid + rank * PA_THREADS; i < A.r * D; i += PA_THREADS * size) {
                const int row = i / D, col = i - row * D;
                const float* src = cl + row * MS;
                float m = -INFINITY, acc = 0.f, l = 0.f, lw = 0.f;
                for (uint32_t k0 = 0; k0 < size; k0 += 8) {      // eight CTAs' loads in flight
                    float mk[8], lk[8], wk[8], ok[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t k = min(k0 + i, size - 1);
                        mk[i] = ld_cluster_f32(src + D, k);
                        lk[i] = ld_cluster_f32(src + D + 1, k);
                        wk[i] = ld_cluster_f32(src + D + 2, k);
                        ok[i] = ld_cluster_f32(src + col, k);
                    }
                    float to = m;
#pragma unroll
                    for (int i = 0; i < 8; ++i) to = fmaxf(to, mk[i]);
                    const float f0 = l == 0.f ? 0.f : ex2(m - to);
                    m = to;
                    l *= f0; lw *= f0; acc *= f0;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k0 + i < size && lk[i] != 0.f) {
                            const float f = ex2(mk[i] - m);
                            l += f * lk[i]; lw += f * wk[i]; acc += f * ok[i];
                        }
                }
                pa_store(A, (int64_t)g * A.r + row, D, col, acc, m, l, lw);
            }
            cluster_barrier();     // nobody leaves while its states are read
            return;
        }
        if (tid == 0 && t0 == 0) {
            // the CTA that holds the group's last tile: the largest c with total * c / n_cta <= that tile
            const long long last = gpre + n - 1;
            long long cl = last * n_cta / total;
            while (cl + 1 < n_cta && total * (cl + 1) / n_cta <= last) ++cl;
            while (cl > 0 && total * cl / n_cta > last) --cl;
            A.info[g] = whole ? make_int2(-1, -1) : make_int2(slot, (int)cl);
        }
        fence_async();             // the next segment's copies overwrite the states
        __syncthreads();
        cur = gpre + t1;
        ++seg;
    }
}

// Joins the parts of groups cut by range borders: grid (G, r); thread (slice, value column), the slices take every
// PA_JOIN-th part and are added in order.
constexpr int PA_JOIN = 4;
template <int D>
__global__ void __launch_bounds__(D * PA_JOIN) paged_join_kernel(const __grid_constant__ PagedAttnArgs A) {
    __shared__ float s_red[D * PA_JOIN / 32];
    __shared__ float s_acc[PA_JOIN][D + 2];
    const int g = blockIdx.x, row = blockIdx.y, col = threadIdx.x % D, slice = threadIdx.x / D;
    grid_wait();
    const int2 info = A.info[g];
    if (info.x < 0) return;
    const int n = info.y - info.x / 2 + 1;                    // parts: the first CTA's slot, then slot 0 of each CTA after it
    auto part = [&](int i) { return (i == 0 ? (int64_t)info.x : 2 * ((int64_t)(info.x / 2) + i)) * A.r + row; };
    float m = -INFINITY;
    for (int i = threadIdx.x; i < n; i += D * PA_JOIN) m = fmaxf(m, A.part_ml[part(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < D * PA_JOIN / 32; ++i) m = fmaxf(m, s_red[i]);
    float acc = 0.f, l = 0.f, lw = 0.f;
#pragma unroll 8
    for (int i = slice; i < n; i += PA_JOIN) {
        const int64_t at = part(i);
        const float4 ml = A.part_ml[at];
        const float o = A.part_o[at * D + col];
        const float f = ex2(ml.x - m);
        // an empty part adds nothing, whatever its maximum
        if (ml.y != 0.f) { l += f * ml.y; lw += f * ml.z; acc += f * o; }
    }
    s_acc[slice][col] = acc;
    if (col == 0) { s_acc[slice][D] = l; s_acc[slice][D + 1] = lw; }
    __syncthreads();
    if (slice) return;
    for (int k = 1; k < PA_JOIN; ++k) acc += s_acc[k][col];
    l = lw = 0.f;
    for (int k = 0; k < PA_JOIN; ++k) { l += s_acc[k][D]; lw += s_acc[k][D + 1]; }
    pa_store(A, (int64_t)g * A.r + row, D, col, acc, m, l, lw);
}

// How a call is cut.
// cluster > 0: that many CTAs per group in a cluster and no second launch.  Taken where a CTA then has at most 2048
// tokens, i.e. where latency counts (1 x 4096 bf16: 6.6 us against 10.9 in two launches), and for lists of blocks,
// whose groups all have the same work (8 x 72 blocks of 64, e4m3: 20.6 us against 26.6).
// cluster 0: equal ranges over `ctas` CTAs, enough to fill the device, at least 8 subtiles each at the lengths the
// caller bounds.  Taken for long contexts, whose lengths the host does not know: where they differ by two a cluster
// per group waits for the longest (16 x 64K-128K e4m3: 455 us against 555).
struct PaPlan {
    int cluster, ctas;
};
constexpr int PA_SLOTS = PA_PER_SM * 152;
PaPlan paged_attn_plan(int64_t groups, int64_t max_tokens, bool equal) {
    const int64_t want = std::max<int64_t>(1, (max_tokens + 127) / 128);
    const int64_t fit = std::min<int64_t>(16, PA_SLOTS / groups);
    const int64_t s = std::max<int64_t>(1, std::min(want, fit));
    if (max_tokens <= 2048 * s || (equal && s * groups >= PA_SLOTS / 2)) return {(int)s, (int)(s * groups)};
    const int64_t subs = groups * ((max_tokens + PA_SUB - 1) / PA_SUB);
    return {0, (int)std::min<int64_t>(PA_SLOTS, std::max<int64_t>(1, (subs + 7) / 8))};
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

size_t paged_attn_workspace(const PaPlan& plan, int G, int r, int d) {
    if (plan.cluster) return 0;
    const int ctas = plan.ctas;
    return round256((size_t)G * sizeof(int2)) + round256((size_t)2 * ctas * r * sizeof(float4)) +
           (size_t)2 * ctas * r * d * sizeof(float);
}

}  // namespace kvo

namespace {

int64_t paged_attn_bound(const kvo_paged_cache* c, int n_blocks, int64_t max_len) {
    const int64_t cap = (int64_t)c->max_pages * c->page_size;
    int64_t n = max_len > 0 && max_len < cap ? max_len : cap;
    if (n_blocks > 0) n = (int64_t)n_blocks * c->page_size;
    return n;
}

const char* paged_attn_error(const kvo_paged_cache* c, int n_q_heads, int n_blocks, int64_t max_len) {
    if (const char* m = kvo::paged_cache_error(c)) return m;
    if (n_q_heads < c->n_kv_heads || n_q_heads % c->n_kv_heads) return "n_q_heads must be a multiple of n_kv_heads";
    if (n_q_heads / c->n_kv_heads > 16) return "n_q_heads / n_kv_heads must be <= 16";
    if (max_len < 0) return "max_len must be >= 0";
    if (n_blocks < 0 || (int64_t)n_blocks * c->page_size >= (1 << 30)) return "n_blocks * page_size must fit in 30 bits";
    return nullptr;
}

template <int D, bool FP8, int NH>
cudaError_t paged_attn_launch(const CUtensorMap& mk, const CUtensorMap& mv, const kvo::PagedAttnArgs& A,
                              const kvo::PaPlan& plan, cudaStream_t s) {
    using namespace kvo;
    const int smem = PA_RING + 1024;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = cudaSuccess;
    if (first_on_device(done)) {
        e = cudaFuncSetAttribute(paged_attn_kernel<D, FP8, NH, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(paged_attn_kernel<D, FP8, NH, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(paged_attn_kernel<D, FP8, NH, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        mark_on_device(done);
    }
    if (plan.cluster)
        return launch_dependent(paged_attn_kernel<D, FP8, NH, true>, plan.ctas, PA_THREADS, smem, s, plan.cluster, mk, mv, A);
    e = launch_dependent(paged_attn_kernel<D, FP8, NH, false>, plan.ctas, PA_THREADS, smem, s, 0, mk, mv, A);
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_join_kernel<D>, dim3(A.G, A.r), D * PA_JOIN, 0, s, 0, A);
}

}  // namespace

extern "C" kvo_status kvo_paged_attn_workspace(const kvo_paged_cache* cache, int n_q_heads, int n_blocks,
                                               int64_t max_len, size_t* bytes_out) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (!bytes_out) return bad("null output pointer");
    *bytes_out = 0;
    if (const char* m = paged_attn_error(cache, n_q_heads, n_blocks, max_len)) return bad(m);
    const int G = cache->batch * cache->n_kv_heads;
    *bytes_out = paged_attn_workspace(paged_attn_plan(std::max(G, 1), paged_attn_bound(cache, n_blocks, max_len), n_blocks > 0), G,
                                      n_q_heads / cache->n_kv_heads, cache->head_dim);
    return KVO_OK;
}

extern "C" kvo_status kvo_paged_attn(const kvo_paged_cache* cache, const void* q, int n_q_heads, const int32_t* lens,
                                     int64_t max_len, const int32_t* blocks, const int32_t* counts, int n_blocks,
                                     void* o, float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                                     kvo_stream_t stream) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (const char* m = paged_attn_error(cache, n_q_heads, blocks ? n_blocks : 0, max_len)) return bad(m);
    if (cache->batch == 0) return KVO_OK;
    if (!q || !lens || !o || !lse) return bad("null pointer argument");
    if (blocks && n_blocks < 1) return bad("blocks needs n_blocks >= 1");
    if (counts && !blocks) return bad("counts needs blocks");
    if ((uintptr_t)q % 16 || (uintptr_t)o % 16 || (uintptr_t)workspace % 256)
        return bad("q and o must be 16-byte aligned, the workspace 256-byte aligned");
    const int G = cache->batch * cache->n_kv_heads, r = n_q_heads / cache->n_kv_heads, D = cache->head_dim;
    const PaPlan plan = paged_attn_plan(G, paged_attn_bound(cache, blocks ? n_blocks : 0, max_len), blocks != nullptr);
    const size_t need = paged_attn_workspace(plan, G, r, D);
    if (need && (!workspace || workspace_bytes < need)) return bad("the workspace is too small (kvo_paged_attn_workspace)");
    const bool fp8 = cache->format == KVO_PAGES_E4M3;
    const int rb = fp8 ? D : 2 * D;
    CUtensorMap mk, mv;
    const uint64_t rows = (uint64_t)cache->n_pages * cache->n_kv_heads * cache->page_size;
    if (!tensor_map_rows(&mk, cache->k_pages, fp8 ? 1 : 2, D, rows, rb > 128 ? 128 : rb, PA_SUB) ||
        !tensor_map_rows(&mv, cache->v_pages, fp8 ? 1 : 2, D, rows, rb > 128 ? 128 : rb, PA_SUB)) {
        set_last_error("cuTensorMapEncodeTiled failed for the pages");
        return KVO_ERR_CUDA;
    }
    PagedAttnArgs A{};
    A.q = (const uint16_t*)q;
    A.scale[0] = fp8 ? cache->k_scale : nullptr;
    A.scale[1] = fp8 ? cache->v_scale : nullptr;
    A.table = cache->table;
    A.lens = lens;
    A.blocks = blocks;
    A.counts = counts;
    A.o = (uint16_t*)o;
    A.lse = lse;
    uint8_t* ws = (uint8_t*)workspace;
    A.info = (int2*)ws;
    A.part_ml = (float4*)(ws + round256((size_t)G * sizeof(int2)));
    A.part_o = (float*)((uint8_t*)A.part_ml + round256((size_t)2 * plan.ctas * r * sizeof(float4)));
    A.status = status;
    A.batch = cache->batch;
    A.hkv = cache->n_kv_heads;
    A.r = r;
    A.page = cache->page_size;
    A.shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : cache->page_size == 64 ? 6 : 7;
    A.n_pages = cache->n_pages;
    A.max_pages = cache->max_pages;
    A.n_blocks = n_blocks;
    A.G = G;
    A.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    A.wait_ns = 2000000000LL;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
#define KVO_PAGED(D_, F_) (r <= 8 ? paged_attn_launch<D_, F_, 1>(mk, mv, A, plan, s) : paged_attn_launch<D_, F_, 2>(mk, mv, A, plan, s))
    if (D == 128) e = fp8 ? KVO_PAGED(128, true) : KVO_PAGED(128, false);
    else e = fp8 ? KVO_PAGED(64, true) : KVO_PAGED(64, false);
#undef KVO_PAGED
    if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    return KVO_OK;
}
