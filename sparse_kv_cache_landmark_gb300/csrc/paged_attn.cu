// kvo_paged_attn: decode attention of one query token per request over a paged
// cache (bf16, or e4m3 with a scale per page and KV head).
//
//   o_h = sum_t softmax_t(q_h . k_t / sqrt(d)) v_t over the tokens of the
//   request (or of the listed blocks of its KV head), lse_h the natural log of
//   the softmax's denominator.
//
// Bound by HBM: each KV head's bytes are read once for all r query heads of
// its group.  Work: the 16-token tiles of every (request, KV head), laid out
// group after group, are cut into equal contiguous ranges, one per CTA (the
// lengths are device data, so each CTA finds its own range by a prefix sum);
// ragged batches therefore end together.  Within a range a group's tiles are
// split over the CTA's four warps; each warp keeps its next tiles in flight in
// its own ring of shared-memory stages, filled by TMA (128-byte-swizzled boxes
// of 16 rows, so that both the key and the value fragments are read without
// bank conflicts).  One pass: running maximum and sum in fp32 registers.
//
// Tensor cores: mma.sync m16n8k16 with the r <= 16 query heads as rows.  e4m3
// codes are widened exactly to f16; q is scaled by a power of two per row so
// that it is exact in f16 as well down to 2^-32 of its row's largest value.
// The weights exp2(s - m) are rounded to f16 (11 bits; bf16 next to bf16
// values, which have a wider exponent than f16) and their sum is taken before
// the rounding, in fp32.  The maximum is only raised when a score passes it by
// more than 2^8, so most tiles have no cross-lane step at all.
//
// A group cut by range borders leaves partial (m, l, o) in the workspace, in
// fp32, joined by a second kernel in a fixed order: results do not depend on
// timing.
#include <cuda.h>
#include <stdio.h>

#include <algorithm>

#include "paged.cuh"
#include "tma_ptx.cuh"
#include "tensor_map.cuh"

namespace kvo {

constexpr int PA_WARPS = 4;
constexpr int PA_THREADS = PA_WARPS * 32;
constexpr int PA_TILE = 16;
constexpr int PA_RING = 64 * 1024;            // bytes of stages per CTA
constexpr float PA_RAISE = 8.f;               // log2: how far a score may pass the running maximum
constexpr float PA_BIAS = 6.f;                // log2: weights are held times 2^6 (f16's small end is 2^-24)

template <int D, bool FP8>
struct PaShape {
    static constexpr int RB = FP8 ? D : 2 * D;               // bytes of a row
    static constexpr int BOX = RB > 128 ? 128 : RB;          // bytes of a box row
    static constexpr int NBOX = RB / BOX;
    static constexpr int TILE_BYTES = PA_TILE * RB;          // K or V of one tile
    static constexpr int STAGE = 2 * TILE_BYTES;
    static constexpr int STAGES = PA_RING / (PA_WARPS * STAGE);
    static constexpr int KCH = RB / 64;                      // 16-byte chunks of a key row per lane
    static constexpr int STEPS = D / 16;                     // k steps of q . k
    static constexpr int NT = D / 8;                         // n tiles of p v
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
    float* part_ml;               // [2 ctas][r][2]
    int2* info;                   // [G]: first and last CTA of a group cut by range borders; x < 0: not cut
    int32_t* status;
    int batch, hkv, r, page, page_tiles, n_pages, max_pages, n_blocks, G;
    float scale_log2;
    long long wait_ns;
};

__device__ __forceinline__ int pa_len(const PagedAttnArgs& A, int b) {
    return min(max(A.lens[b], 0), A.max_pages * A.page);
}
// 16-token tiles of group g
__device__ __forceinline__ int pa_tiles(const PagedAttnArgs& A, int g) {
    if (A.blocks) {
        const int n = A.counts ? min(max(A.counts[g], 0), A.n_blocks) : A.n_blocks;
        return n * A.page_tiles;
    }
    return (pa_len(A, g / A.hkv) + PA_TILE - 1) / PA_TILE;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
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

// One warp's running state for the group's 16 query rows; lane (g, c) = (lane / 4,
// lane % 4) holds rows g and g + 8: o[j] covers value columns col(j, 2c), col(j, 2c + 1).
template <int D, bool FP8>
struct PaState {
    using S = PaShape<D, FP8>;
    float o[S::NT][4];
    float m[2], l[2];              // l: this lane's share of the sum
    float vs;                      // the value scale that o is held in
};

// Scores and values of one tile of 16 tokens, nv of them (1..16) real.
template <int D, bool FP8>
__device__ __forceinline__ void pa_tile(PaState<D, FP8>& T, const uint32_t (&qf)[PaShape<D, FP8>::STEPS][4],
                                        const float (&qs)[2], uint32_t ks, uint32_t vsm, float kscale, float vscale,
                                        int nv) {
    using S = PaShape<D, FP8>;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float sc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
        const int row = 8 * i + g;
#pragma unroll
        for (int m = 0; m < S::KCH; ++m) {
            uint32_t a;
            if (S::BOX == 128) a = ks + (m >> 1) * (PA_TILE * 128) + row * 128 + (((2 * c + (m & 1)) ^ (row & 7)) << 4);
            else a = ks + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
            const uint4 v = lds128(a);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (FP8) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma16816<FP8>(sc[i], qf[4 * m + s], e4m3x2_to_f16x2((uint16_t)w[s]),
                                  e4m3x2_to_f16x2((uint16_t)(w[s] >> 16)));
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s) mma16816<FP8>(sc[i], qf[2 * m + s], w[2 * s], w[2 * s + 1]);
            }
        }
    }
    const float f0 = qs[0] * kscale, f1 = qs[1] * kscale;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sc[i][0] *= f0; sc[i][1] *= f0; sc[i][2] *= f1; sc[i][3] *= f1;
    }
    if (nv < PA_TILE) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (8 * i + 2 * c + (e & 1) >= nv) sc[i][e] = -INFINITY;
    }
    float mx[2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
        mx[x] = fmaxf(fmaxf(sc[0][2 * x], sc[0][2 * x + 1]), fmaxf(sc[1][2 * x], sc[1][2 * x + 1]));
    if (__any_sync(0xffffffffu, mx[0] > T.m[0] + PA_RAISE || mx[1] > T.m[1] + PA_RAISE)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
            mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
            const float m = fmaxf(T.m[x], mx[x]);
            const float f = T.m[x] == -INFINITY ? 0.f : ex2(T.m[x] - m);
            T.m[x] = m;
            T.l[x] *= f;
#pragma unroll
            for (int j = 0; j < S::NT; ++j) { T.o[j][2 * x] *= f; T.o[j][2 * x + 1] *= f; }
        }
    }
    float fold = 1.f;              // what a weight is multiplied by so that o stays in units of T.vs
    if (FP8) {
        if (vscale > T.vs) {       // uniform over the warp
            const float f = T.vs / vscale;
            T.vs = vscale;
#pragma unroll
            for (int j = 0; j < S::NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) T.o[j][e] *= f;
        }
        if (vscale != T.vs) fold = vscale / T.vs;
    }
    const float b0 = PA_BIAS - (T.m[0] == -INFINITY ? 0.f : T.m[0]), b1 = PA_BIAS - (T.m[1] == -INFINITY ? 0.f : T.m[1]);
    float p[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        p[i][0] = ex2(sc[i][0] + b0); p[i][1] = ex2(sc[i][1] + b0);
        p[i][2] = ex2(sc[i][2] + b1); p[i][3] = ex2(sc[i][3] + b1);
        T.l[0] += p[i][0] + p[i][1];
        T.l[1] += p[i][2] + p[i][3];
    }
    uint32_t pa[4];
    if (FP8) {
        pa[0] = pack_f16(p[0][0] * fold, p[0][1] * fold); pa[1] = pack_f16(p[0][2] * fold, p[0][3] * fold);
        pa[2] = pack_f16(p[1][0] * fold, p[1][1] * fold); pa[3] = pack_f16(p[1][2] * fold, p[1][3] * fold);
    } else {
        pa[0] = pack_bf(p[0][0], p[0][1]); pa[1] = pack_bf(p[0][2], p[0][3]);
        pa[2] = pack_bf(p[1][0], p[1][1]); pa[3] = pack_bf(p[1][2], p[1][3]);
    }
    // values: this lane's token rows 2c, 2c + 1, 2c + 8, 2c + 9
    const int tr[4] = {2 * c, 2 * c + 1, 2 * c + 8, 2 * c + 9};
    constexpr int VCH = S::NBOX;                             // 16-byte chunks of a value row per lane (8 bytes: d 64 in e4m3)
    constexpr int VW = S::RB == 64 ? 2 : 4;                  // 32-bit words of a chunk
#pragma unroll
    for (int e = 0; e < VCH; ++e) {
        uint32_t w[4][VW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (S::BOX == 128) {
                const uint4 v = lds128(vsm + e * (PA_TILE * 128) + tr[k] * 128 + ((g ^ (tr[k] & 7)) << 4));
                w[k][0] = v.x; w[k][1] = v.y; w[k][VW - 2] = v.z; w[k][VW - 1] = v.w;
            } else {
                const uint2 v = lds64(vsm + tr[k] * 64 + ((((g >> 1) ^ ((tr[k] >> 1) & 3)) << 4) | ((g & 1) << 3)));
                w[k][0] = v.x; w[k][1] = v.y;
            }
        }
        if (nv < PA_TILE) {        // rows past the end hold anything, NaN included: 0 * NaN must not reach o
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (tr[k] >= nv)
#pragma unroll
                    for (int i = 0; i < VW; ++i) w[k][i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            if (FP8) {             // 4 columns a word
                const uint32_t x0 = __byte_perm(w[0][i], w[1][i], 0x5140), x1 = __byte_perm(w[2][i], w[3][i], 0x5140);
                const uint32_t y0 = __byte_perm(w[0][i], w[1][i], 0x7362), y1 = __byte_perm(w[2][i], w[3][i], 0x7362);
                const int j = (e * VW + i) * 4;
                mma16816<FP8>(T.o[j], pa, e4m3x2_to_f16x2((uint16_t)x0), e4m3x2_to_f16x2((uint16_t)x1));
                mma16816<FP8>(T.o[j + 1], pa, e4m3x2_to_f16x2((uint16_t)(x0 >> 16)), e4m3x2_to_f16x2((uint16_t)(x1 >> 16)));
                mma16816<FP8>(T.o[j + 2], pa, e4m3x2_to_f16x2((uint16_t)y0), e4m3x2_to_f16x2((uint16_t)y1));
                mma16816<FP8>(T.o[j + 3], pa, e4m3x2_to_f16x2((uint16_t)(y0 >> 16)), e4m3x2_to_f16x2((uint16_t)(y1 >> 16)));
            } else {               // 2 columns a word
                const int j = (e * VW + i) * 2;
                mma16816<FP8>(T.o[j], pa, __byte_perm(w[0][i], w[1][i], 0x5410), __byte_perm(w[2][i], w[3][i], 0x5410));
                mma16816<FP8>(T.o[j + 1], pa, __byte_perm(w[0][i], w[1][i], 0x7632), __byte_perm(w[2][i], w[3][i], 0x7632));
            }
        }
    }
}

// Value column of accumulator j at fragment column n (0..7).
template <int D, bool FP8>
__device__ __forceinline__ int pa_col(int j, int n) {
    if (FP8) return n * (D / 8) + j;
    return (j >> 3) * 64 + n * 8 + (j & 7);
}

// What one lane knows of a batch of 32 pages of the segment: page, scales, tokens.
struct PaPage {
    int row;          // first row of the page in the pool seen as [n_pages * Hkv * page] rows; < 0: skip
    int tokens;       // real tokens of the page
    float ks, vs;
};

__device__ __forceinline__ PaPage pa_page(const PagedAttnArgs& A, int g, int i, int len, int n_logical) {
    PaPage P{-1, 0, 1.f, 1.f};
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
    }
    return P;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(PA_THREADS, 3)
paged_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ PagedAttnArgs A) {
    using S = PaShape<D, FP8>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[PA_WARPS * S::STAGES];
    __shared__ long long s_pre;
    __shared__ int s_g, s_dead;
    __shared__ long long s_scan[PA_THREADS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    float* mrg = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) + PA_RING);   // [4][r][D + 3]
    const int MS = D + 3;
    const uint32_t wring = ring + warp * S::STAGES * S::STAGE;
    const uint32_t wbar = smem_u32(bars) + warp * S::STAGES * 8;
    if (lane == 0)
        for (int i = 0; i < S::STAGES; ++i) mbar_init(wbar + 8 * i, 1);
    if (tid == 0) s_dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

    // this CTA's range of the tiles of all groups
    const int per = (A.G + PA_THREADS - 1) / PA_THREADS;
    long long sum = 0;
    for (int i = 0; i < per; ++i) {
        const int g = tid * per + i;
        if (g >= A.G) break;
        sum += pa_tiles(A, g);
        const int len = A.lens[g / A.hkv];
        const bool bad_count = A.counts && (A.counts[g] < 0 || A.counts[g] > A.n_blocks);
        if (blockIdx.x == 0 && A.status && (len < 0 || len > (int64_t)A.max_pages * A.page || bad_count))
            atomicOr(A.status, KVO_DEV_BAD_COUNT);
    }
    s_scan[tid] = sum;
    __syncthreads();
    for (int o = 1; o < PA_THREADS; o <<= 1) {
        const long long x = tid >= o ? s_scan[tid - o] : 0;
        __syncthreads();
        s_scan[tid] += x;
        __syncthreads();
    }
    const long long pre = s_scan[tid] - sum, total = s_scan[PA_THREADS - 1];
    const long long n_cta = max(1ll, min((long long)gridDim.x, total));      // a tile for each, so every range holds work
    const long long lo = blockIdx.x < n_cta ? total * blockIdx.x / n_cta : total;
    const long long hi = blockIdx.x < n_cta ? total * (blockIdx.x + 1) / n_cta : total;
    if (lo >= pre && lo < pre + sum) {
        long long at = pre;
        for (int i = 0; i < per; ++i) {
            const int g = tid * per + i;
            const int n = g < A.G ? pa_tiles(A, g) : 0;
            if (lo < at + n) { s_g = g; s_pre = at; break; }
            at += n;
        }
    }
    __syncthreads();
    // groups with nothing to attend to (and the cut marks of all groups: the CTA with a group's first tile sets it)
    for (int g = blockIdx.x; g < A.G; g += gridDim.x)
        if (pa_tiles(A, g) == 0) {
            for (int i = tid; i < A.r * D; i += PA_THREADS) A.o[(int64_t)g * A.r * D + i] = 0;
            for (int i = tid; i < A.r; i += PA_THREADS) A.lse[(int64_t)g * A.r + i] = -INFINITY;
            if (tid == 0) A.info[g] = make_int2(-1, -1);
        }
    if (lo >= hi) return;

    uint32_t phase = 0;            // bit i: parity of stage i's next wait
    long long cur = lo, gpre = s_pre;
    int g = s_g, seg = 0;
    bool dead = false;
    while (cur < hi) {
        int n = pa_tiles(A, g);
        if (cur >= gpre + n) { gpre += n; ++g; continue; }
        const int t0 = (int)(cur - gpre), t1 = (int)min((long long)n, hi - gpre);
        const int len = pa_len(A, g / A.hkv);
        const int n_logical = A.blocks ? n / A.page_tiles : (len + A.page - 1) / A.page;
        // this warp's tiles
        const int w0 = t0 + (int)((long long)(t1 - t0) * warp / PA_WARPS);
        const int w1 = t0 + (int)((long long)(t1 - t0) * (warp + 1) / PA_WARPS);

        // query fragments: rows g and g + 8 of the group (heads beyond r: zero)
        uint32_t qf[S::STEPS][4];
        float qs[2];
        {
            const int gr = lane >> 2, c = lane & 3;
            const uint16_t* qg = A.q + (int64_t)g * A.r * D;
            float amax[2] = {0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = gr + 8 * x;
#pragma unroll
                for (int m = 0; m < S::KCH; ++m) {
                    constexpr int ES = FP8 ? 1 : 2;
                    const int box = S::BOX == 128 ? m >> 1 : 0, ch = S::BOX == 128 ? 2 * c + (m & 1) : c;
                    const int e0 = box * (128 / ES) + ch * (16 / ES);
                    constexpr int PER = FP8 ? 4 : 2;         // steps of a chunk
#pragma unroll
                    for (int s = 0; s < PER; ++s)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t v = row < A.r ? *reinterpret_cast<const uint32_t*>(qg + row * D + e0 + 4 * s + 2 * k) : 0u;
                            qf[PER * m + s][x + 2 * k] = v;
                            amax[x] = fmaxf(amax[x], fmaxf(fabsf(bf16lo_to_f32(v)), fabsf(bf16hi_to_f32(v))));
                        }
                }
                qs[x] = A.scale_log2;
                if (FP8) {
                    amax[x] = fmaxf(amax[x], __shfl_xor_sync(0xffffffffu, amax[x], 1));
                    amax[x] = fmaxf(amax[x], __shfl_xor_sync(0xffffffffu, amax[x], 2));
                    // row / 2^(e - 8): the largest value is in [2^8, 2^9)
                    const int e = min(max((int)(__float_as_uint(amax[x]) >> 23) - 127, -110), 126);
                    const float f = __uint_as_float((uint32_t)(8 - e + 127) << 23);
                    qs[x] = A.scale_log2 * __uint_as_float((uint32_t)(e - 8 + 127) << 23);
#pragma unroll
                    for (int s = 0; s < S::STEPS; ++s)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t v = qf[s][x + 2 * k];
                            qf[s][x + 2 * k] = pack_f16(bf16lo_to_f32(v) * f, bf16hi_to_f32(v) * f);
                        }
                }
            }
        }
        PaState<D, FP8> T;
#pragma unroll
        for (int j = 0; j < S::NT; ++j) T.o[j][0] = T.o[j][1] = T.o[j][2] = T.o[j][3] = 0.f;
        T.m[0] = T.m[1] = -INFINITY;
        T.l[0] = T.l[1] = 0.f;
        T.vs = 0.f;

        // tiles w0..w1: pages come in batches of 32, one per lane; the next batch is loaded while this one is used
        int base = w0 / A.page_tiles;
        PaPage cur_p = pa_page(A, g, base + lane, len, n_logical), nxt_p = pa_page(A, g, base + 32 + lane, len, n_logical);
        int issued = w0;
        auto issue = [&](int t) {  // copies of tile t into its stage
            const int pg = t / A.page_tiles, k = pg - base;
            const int src_row = k < 32 ? __shfl_sync(0xffffffffu, cur_p.row, k & 31) : __shfl_sync(0xffffffffu, nxt_p.row, k & 31);
            const int src_tok = k < 32 ? __shfl_sync(0xffffffffu, cur_p.tokens, k & 31) : __shfl_sync(0xffffffffu, nxt_p.tokens, k & 31);
            const int off = (t - pg * A.page_tiles) * PA_TILE;
            const int st = (t - w0) % S::STAGES;
            if (lane == 0 && src_row >= 0 && off < src_tok) {
                const uint32_t bar = wbar + 8 * st, dst = wring + st * S::STAGE;
                mbar_expect_tx(bar, S::STAGE);
#pragma unroll
                for (int x = 0; x < S::NBOX; ++x) {
                    tma_load_2d(dst + x * (PA_TILE * 128), &map_k, x * (128 / (FP8 ? 1 : 2)), src_row + off, bar);
                    tma_load_2d(dst + S::TILE_BYTES + x * (PA_TILE * 128), &map_v, x * (128 / (FP8 ? 1 : 2)), src_row + off, bar);
                }
            }
        };
        for (; issued < min(w1, w0 + S::STAGES); ++issued) issue(issued);
        // Every copy issued is waited for, also after a wait that ran out: none may land once the CTA has left.
        for (int t = w0; t < issued; ++t) {
            const int pg = t / A.page_tiles;
            if (pg - base >= 32) {
                base += 32;
                cur_p = nxt_p;
                nxt_p = pa_page(A, g, base + 32 + lane, len, n_logical);
            }
            const int k = pg - base;
            const int row = __shfl_sync(0xffffffffu, cur_p.row, k), tok = __shfl_sync(0xffffffffu, cur_p.tokens, k);
            const float ks = __shfl_sync(0xffffffffu, cur_p.ks, k), vs = __shfl_sync(0xffffffffu, cur_p.vs, k);
            const int nv = min(PA_TILE, tok - (t - pg * A.page_tiles) * PA_TILE);
            const int st = (t - w0) % S::STAGES;
            if (row >= 0 && nv > 0) {
                if (!mbar_wait_bounded(wbar + 8 * st, (phase >> st) & 1, A.wait_ns)) dead = true;
                phase ^= 1u << st;
                if (!dead) pa_tile<D, FP8>(T, qf, qs, wring + st * S::STAGE, wring + st * S::STAGE + S::TILE_BYTES, ks, vs, nv);
            }
            dead = __any_sync(0xffffffffu, dead);
            if (issued < w1 && !dead) issue(issued++);
        }
        if (dead) {                // a copy never came: say so, and leave once every thread knows
            if (lane == 0) { if (A.status) atomicOr(A.status, KVO_DEV_TIMEOUT); s_dead = 1; }
        }
        // the warps' states
        {
            const int gr = lane >> 2, c = lane & 3;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float l = T.l[x];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                const int row = gr + 8 * x;
                if (row < A.r) {
                    float* dst = mrg + (warp * A.r + row) * MS;
                    if (c == 0) { dst[D] = T.m[x]; dst[D + 1] = l; dst[D + 2] = FP8 ? T.vs : 1.f; }
#pragma unroll
                    for (int j = 0; j < S::NT; ++j) {
                        dst[pa_col<D, FP8>(j, 2 * c)] = T.o[j][2 * x];
                        dst[pa_col<D, FP8>(j, 2 * c + 1)] = T.o[j][2 * x + 1];
                    }
                }
            }
        }
        __syncthreads();
        if (s_dead) return;
        const bool whole = t0 == 0 && t1 == n;
        const int slot = 2 * blockIdx.x + (seg ? 1 : 0);
        for (int i = tid; i < A.r * D; i += PA_THREADS) {
            const int row = i / D, col = i - row * D;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < PA_WARPS; ++w) m = fmaxf(m, mrg[(w * A.r + row) * MS + D]);
            float acc = 0.f, l = 0.f;
#pragma unroll
            for (int w = 0; w < PA_WARPS; ++w) {
                const float* src = mrg + (w * A.r + row) * MS;
                if (src[D + 1] == 0.f) continue;
                const float f = ex2(src[D] - m);
                l += f * src[D + 1];
                acc += f * src[D + 2] * src[col];
            }
            if (whole) {
                const int64_t at = (int64_t)g * A.r + row;
                A.o[at * D + col] = __bfloat16_as_ushort(__float2bfloat16_rn(l != 0.f ? acc / l : 0.f));
                if (col == 0) A.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l) - PA_BIAS) * 0.6931471805599453f;
            } else {
                const int64_t at = (int64_t)slot * A.r + row;
                A.part_o[at * D + col] = acc;
                if (col == 0) { A.part_ml[2 * at] = m; A.part_ml[2 * at + 1] = l; }
            }
        }
        if (tid == 0 && t0 == 0) {
            // the CTA that holds the group's last tile: the largest c with total * c / n_cta <= that tile
            const long long last = gpre + n - 1;
            long long cl = last * n_cta / total;
            while (cl + 1 < n_cta && total * (cl + 1) / n_cta <= last) ++cl;
            while (cl > 0 && total * cl / n_cta > last) --cl;
            A.info[g] = whole ? make_int2(-1, -1) : make_int2(2 * (int)blockIdx.x + (seg ? 1 : 0), (int)cl);
        }
        __syncthreads();
        cur = gpre + t1;
        ++seg;
    }
}

// Joins the parts of groups cut by range borders: grid (G, r), one thread per value column.
template <int D>
__global__ void __launch_bounds__(D) paged_join_kernel(const __grid_constant__ PagedAttnArgs A) {
    const int g = blockIdx.x, row = blockIdx.y, col = threadIdx.x;
    const int2 info = A.info[g];
    if (info.x < 0) return;
    const int n = info.y - info.x / 2 + 1;                    // parts: the first CTA's slot, then slot 0 of each CTA after it
    auto part = [&](int i) { return i == 0 ? (int64_t)info.x : 2 * ((int64_t)(info.x / 2) + i); };
    float m = -INFINITY;
    for (int i = 0; i < n; ++i) m = fmaxf(m, A.part_ml[2 * (part(i) * A.r + row)]);
    float acc = 0.f, l = 0.f;
    for (int i = 0; i < n; ++i) {
        const int64_t at = part(i) * A.r + row;
        const float li = A.part_ml[2 * at + 1];
        if (li == 0.f) continue;
        const float f = ex2(A.part_ml[2 * at] - m);
        l += f * li;
        acc += f * A.part_o[at * D + col];
    }
    const int64_t at = (int64_t)g * A.r + row;
    A.o[at * D + col] = __bfloat16_as_ushort(__float2bfloat16_rn(l != 0.f ? acc / l : 0.f));
    if (col == 0) A.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l) - PA_BIAS) * 0.6931471805599453f;
}

// CTAs of the main kernel: enough to fill the device three to an SM, and at
// least 8 tiles (two a warp) each at the lengths the caller bounds.
int paged_attn_ctas(int64_t groups, int64_t max_tokens) {
    const int64_t tiles = groups * ((max_tokens + PA_TILE - 1) / PA_TILE);
    return (int)std::min<int64_t>(3 * 152, std::max<int64_t>(1, (tiles + 7) / 8));
}

size_t paged_attn_workspace(int ctas, int G, int r, int d) {
    const size_t ml = (size_t)2 * ctas * r * 2 * sizeof(float), o = (size_t)2 * ctas * r * d * sizeof(float);
    return ((size_t)G * sizeof(int2) + 255) / 256 * 256 + (ml + 255) / 256 * 256 + o;
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
    if (n_blocks < 0 || (int64_t)n_blocks * c->page_size > INT32_MAX) return "n_blocks * page_size must fit in 31 bits";
    return nullptr;
}

template <int D, bool FP8>
cudaError_t paged_attn_launch(const CUtensorMap& mk, const CUtensorMap& mv, const kvo::PagedAttnArgs& A, int ctas,
                              cudaStream_t s) {
    using namespace kvo;
    const int smem = PA_RING + 1024 + PA_WARPS * A.r * (D + 3) * (int)sizeof(float);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = cudaSuccess;
    if (first_on_device(done)) {
        e = cudaFuncSetAttribute(paged_attn_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PA_RING + 1024 + PA_WARPS * 16 * (D + 3) * (int)sizeof(float));
        if (e != cudaSuccess) return e;
        mark_on_device(done);
    }
    paged_attn_kernel<D, FP8><<<ctas, PA_THREADS, smem, s>>>(mk, mv, A);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    paged_join_kernel<D><<<dim3(A.G, A.r), D, 0, s>>>(A);
    return cudaGetLastError();
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
    *bytes_out = paged_attn_workspace(paged_attn_ctas(G, paged_attn_bound(cache, n_blocks, max_len)), G,
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
    if (!q || !lens || !o || !lse || !workspace) return bad("null pointer argument");
    if (blocks && n_blocks < 1) return bad("blocks needs n_blocks >= 1");
    if (counts && !blocks) return bad("counts needs blocks");
    if ((uintptr_t)q % 16 || (uintptr_t)o % 16 || (uintptr_t)workspace % 256)
        return bad("q and o must be 16-byte aligned, the workspace 256-byte aligned");
    const int G = cache->batch * cache->n_kv_heads, r = n_q_heads / cache->n_kv_heads, D = cache->head_dim;
    const int ctas = paged_attn_ctas(G, paged_attn_bound(cache, blocks ? n_blocks : 0, max_len));
    if (workspace_bytes < paged_attn_workspace(ctas, G, r, D)) return bad("the workspace is too small (kvo_paged_attn_workspace)");
    const bool fp8 = cache->format == KVO_PAGES_E4M3;
    const int rb = fp8 ? D : 2 * D;
    CUtensorMap mk, mv;
    const uint64_t rows = (uint64_t)cache->n_pages * cache->n_kv_heads * cache->page_size;
    if (!tensor_map_rows(&mk, cache->k_pages, fp8 ? 1 : 2, D, rows, rb > 128 ? 128 : rb, PA_TILE) ||
        !tensor_map_rows(&mv, cache->v_pages, fp8 ? 1 : 2, D, rows, rb > 128 ? 128 : rb, PA_TILE)) {
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
    A.part_ml = (float*)(ws + ((size_t)G * sizeof(int2) + 255) / 256 * 256);
    A.part_o = (float*)((uint8_t*)A.part_ml + ((size_t)2 * ctas * r * 2 * sizeof(float) + 255) / 256 * 256);
    A.status = status;
    A.batch = cache->batch;
    A.hkv = cache->n_kv_heads;
    A.r = r;
    A.page = cache->page_size;
    A.page_tiles = cache->page_size / PA_TILE;
    A.n_pages = cache->n_pages;
    A.max_pages = cache->max_pages;
    A.n_blocks = n_blocks;
    A.G = G;
    A.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    A.wait_ns = 2000000000LL;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (D == 128) e = fp8 ? paged_attn_launch<128, true>(mk, mv, A, ctas, s) : paged_attn_launch<128, false>(mk, mv, A, ctas, s);
    else e = fp8 ? paged_attn_launch<64, true>(mk, mv, A, ctas, s) : paged_attn_launch<64, false>(mk, mv, A, ctas, s);
    if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    return KVO_OK;
}
