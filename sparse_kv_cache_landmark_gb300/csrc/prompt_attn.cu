// kvo_prompt_attn: causal (or full) GQA attention over packed prompts.
//
//   o_i = sum_t softmax_t(q_i . k_t / sqrt(d)) v_t,  t <= i + (nk - nq) where causal.
//
// Bound by the tensor cores: 4 d FLOPs for every (query head, visible pair).
//
// A work item is 256 query rows of one KV head: two tiles of 128 rows, each
// floor(128 / r) tokens x the r query heads of the group, so that every K and V
// tile is fetched once for the whole group and short prompts fill their tiles.
// One CTA per item and SM, heaviest items first (or, where few items would leave
// SMs idle, a cluster of 2, 4 or 8 CTAs that split the item's keys and join their
// parts through distributed shared memory, in a fixed order):
//   warp 9   loads Q once and K, V tiles of 128 keys through a ring (TMA),
//   warps 8, 10  one thread each issues the tcgen05.mma of tile 0 and 1: S_t =
//            Q_t K^T (shared x shared) and O_t += P_t V (tensor memory x
//            shared), in the order O_t(j), S_t(j+1): a tile's softmax runs
//            beside the other tile's two products,
//   warps 0-3, 4-7  the softmax of tile 0 and 1, one thread per row: S from
//            tensor memory, online maximum and sum in fp32, P (bf16) back over S.
// Tensor memory (512 columns): S_0, S_1 (128 each, P over their first half),
// O_0, O_1 (d each, fp32).  O is rescaled, by the softmax threads, only when a
// row's maximum rises by more than 2^8 (P then stays below 2^8 and the sum is
// kept in the same units), which after the first tiles is rare.
//
// What bounds it: with P in tensor memory a value product of K = 16 takes 105
// cycles instead of the 64 of its FLOPs (measured alone, at N = 64 and 128 alike),
// so a pair of 128-key tiles takes 2440 cycles of products, 2550 with its two
// commits, against 2048 at full rate; the kernel runs one in 2790.  P in shared
// memory would take 2120, but then products, P and the tiles that arrive ask for
// 3070 cycles of shared-memory bandwidth.  An item's start and end (its first
// loads, its last softmax and rows) add about 5 us, the join of split items 5 more:
// 64 KB of fp32 rows come from the other CTAs' shared memory at about 10 bytes a
// cycle and SM, 3.5 us.
//
// Measured (32 query and 8 KV heads of 128): 16384 tokens 1400 us (1570 TFLOP/s, 0.83
// of cuBLAS's bf16 rate here), 8192 356 us (1540), 3 chunks of 4099 tokens in all
// behind 6000 keys each 335 us (1370: 3.5 waves of items), 13 prompts of 2203
// tokens in all, 8 and 2 heads of 64, 10 us.
//
// The weights P are rounded to bf16 as the matrix instruction takes them (V is
// bf16, both operands have one type); their sum is taken in fp32 before that.
#include <stdio.h>

#include <algorithm>

#include "kvo_internal.cuh"
#include "launch.cuh"
#include "paged.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace kvo {

constexpr int PR_THREADS = 384;
constexpr int PR_ROWS = 128;               // query rows of a tile
constexpr int PR_KEYS = 128;               // keys of a tile
constexpr int PR_BLOCK = PR_ROWS * 128;    // bytes of 128 rows x 64 values
constexpr float PR_RAISE = 8.f;            // log2

template <int D>
struct PrShape {
    static constexpr int TILE = (D / 64) * PR_BLOCK;            // bytes of 128 rows x D values
    static constexpr int STAGES = (192 * 1024 - 2 * TILE) / TILE;
    static constexpr int DEPTH = STAGES / 2;                    // tiles of keys that fit the ring, K and V
    static constexpr int SMEM = (2 + STAGES) * TILE + 1024;     // > half an SM's: one CTA per SM
};

struct PromptArgs {
    const int32_t* cu_q;
    const int32_t* cu_k;
    uint16_t* o;
    float* lse;                    // or NULL
    int32_t* status;
    long long total_q, total_k;
    int batch, hq, hkv, r, tq, causal, units;
    float scale_log2;
    int skip;                      // the load (K(0), V(0), K(1), ..) that every CTA announces without copying it (tests; -1: none)
    long long wait_ns;
};

__device__ __forceinline__ float pr_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

struct PrShared {
    uint64_t q_full[2], kv_full[12], s_full[2][6], p_full[2][2], o_done[2], turn[2], drain[2], v_tail;
    uint32_t tmem;
    int abort;
    int issued, tail_open;         // what the loading warp leaves: its loads, and whether one more is on its way into v_tail
};

// A wait that gives up after the limit, or once another warp has; every caller then leaves its loop.
__device__ __forceinline__ bool pr_wait_long(int* abort, int32_t* status, uint32_t bar, uint32_t parity, long long limit) {
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
__device__ __forceinline__ bool pr_wait(PrShared& sh, const PromptArgs& A, uint64_t& bar, uint32_t parity) {
    const uint32_t b = smem_u32(&bar);
    if (mbar_try_wait(b, parity)) return true;
    return pr_wait_long(&sh.abort, A.status, b, parity, A.wait_ns);
}

// One part of an item: 256 rows of fp32 values in shared memory, each with its maximum and sum.  16-byte chunks, turned
// by the row against bank conflicts.
template <int D>
__device__ __forceinline__ float4* pr_part_row(uint8_t* part, int i, int chunk) {
    return reinterpret_cast<float4*>(part) + i * (D / 4) + (chunk ^ (i & 7));
}
template <int D>
__device__ __forceinline__ float2* pr_part_ml(uint8_t* part, int i) {
    return reinterpret_cast<float2*>(part + 2 * PR_ROWS * D * 4) + i;
}
// The softmax of one tile: a thread owns row `row` of it; the row sees its request's keys [0, limit).
template <int D, bool SPLIT>
__device__ __forceinline__ void pr_softmax(PrShared& sh, const PromptArgs& A, int t, int n_tiles, int limit, bool real,
                                           int64_t out_row, uint8_t* smem) {
    const uint32_t lanes = (uint32_t)(threadIdx.x & 96) << 16;          // this warp's quarter of the lanes
    const uint32_t S = sh.tmem + 128 * t + lanes, O = sh.tmem + 256 + D * t + lanes;
    float m = -INFINITY, l = 0.f;                                       // log2 units; l in units of 2^m
    bool ok = true;
    int slot = 0;                  // of S(j)'s barrier, and its parity
    uint32_t parity = 0;
    for (int j = 0; j < n_tiles; ++j) {
        ok = pr_wait(sh, A, sh.s_full[t][slot], parity);
        if (++slot == PrShape<D>::DEPTH) { slot = 0; parity ^= 1; }
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[PR_KEYS];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(S + 32 * i, s + 32 * i);
        tmem_wait_ld();
        const int rem = limit - j * PR_KEYS;
        if (rem < PR_KEYS) {
#pragma unroll
            for (int i = 0; i < PR_KEYS; ++i)
                if (i >= rem) s[i] = 0xFF800000u;                       // -inf
        }
        float mx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(s[e]);
#pragma unroll
        for (int i = 4; i + 8 <= PR_KEYS; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(s[i + e]), __uint_as_float(s[i + 4 + e]));
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(s[PR_KEYS - 4 + e]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * A.scale_log2;
        if (__any_sync(0xffffffffu, top > m + PR_RAISE)) {
            const float to = fmaxf(m, top);
            const float f = m == -INFINITY ? 0.f : pr_ex2(m - to);
            m = to;
            l *= f;
            if (j > 0) {           // S(j) complete: so is O += P(j - 1) V, which was issued before it
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(O + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    tmem_st32(O + c, o);
                }
            }
        }
        const float b = m == -INFINITY ? 0.f : -m;
        const uint64_t scale2 = pack2(A.scale_log2, A.scale_log2), b2 = pack2(b, b);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(s[32 * h + 2 * i]), __uint_as_float(s[32 * h + 2 * i + 1])), scale2, b2), x, y);
                x = pr_ex2(x);
                y = pr_ex2(y);
                sum[i & 1] = add2(sum[i & 1], pack2(x, y));
                const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
                p[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            tmem_st16(S + 16 * h, p);
            if (h & 1) {           // half of the weights are there: the value product may begin on them
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.p_full[t][h >> 1]));
            }
        }
        float s0, s1;
        unpack2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
    }
    if (ok && n_tiles > 0) {
        ok = pr_wait(sh, A, sh.o_done[t], 0);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
    }
    if constexpr (SPLIT) {
        // Both tiles' products are done: what they read may be overwritten.  After a wait that ran out loads may still land
        // over the parts: the outputs are invalid then, and the loading warp waits for its loads before the CTA leaves.
        bar_named(1, 256);
        const int i = threadIdx.x;
        if (n_tiles > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(O + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *pr_part_row<D>(smem, i, (c + e) / 4) = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                                        __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
            }
        }
        *pr_part_ml<D>(smem, i) = make_float2(m, l);
        return;
    }
    if (!ok) return;
    uint8_t* q_smem = smem + t * PrShape<D>::TILE;
    // The row goes through this warp's part of Q's memory (its tile's products are done), so that the warp writes
    // whole rows: 32 threads with a row each would touch 32 lines a store.  16-byte chunks, turned by the row against
    // bank conflicts.
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int lane = threadIdx.x & 31;
    constexpr int CH = D / 8;                                           // chunks of a row
    uint8_t* rows = q_smem + (threadIdx.x & 96) * (2 * D);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (n_tiles > 0) {
            tmem_ld32(O + c, o);
            tmem_wait_ld();
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // a row that saw nothing is zero, whatever its lane of tensor memory holds
                const float x = l != 0.f ? __uint_as_float(o[i + 2 * e]) * inv : 0.f;
                const float y = l != 0.f ? __uint_as_float(o[i + 2 * e + 1]) * inv : 0.f;
                const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
                w[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            const int ch = ((c + i) / 8) ^ (lane & 7);
            *reinterpret_cast<uint4*>(rows + lane * (2 * D) + ch * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < CH; ++i) {                                      // 32 / CH rows at a time
        const int row = i * (32 / CH) + lane / CH, ch = lane % CH;
        const long long to = __shfl_sync(0xffffffffu, real ? (long long)out_row : -1ll, row);
        const uint4 v = *reinterpret_cast<const uint4*>(rows + row * (2 * D) + (ch ^ (row & 7)) * 16);
        if (to >= 0) *reinterpret_cast<uint4*>(A.o + to * D + ch * 8) = v;
    }
    if (real && A.lse) A.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Joins the parts of an item: this CTA takes every PARTS-th row.  A warp's lanes hold AT_ONCE rows; BATCH of those are
// fetched together, since each takes the way to the other CTAs' shared memory and back.
template <int D, int PARTS>
__device__ __forceinline__ void pr_join(const PromptArgs& A, uint8_t* smem, int part, int g, int64_t qs, int nq, int tok0) {
    constexpr int CH = D / 4, AT_ONCE = 32 / CH, ROWS = 2 * PR_ROWS / PARTS / 8, TURNS = ROWS / AT_ONCE;
    constexpr int BATCH = TURNS < 16 / PARTS ? TURNS : 16 / PARTS;
    static_assert(ROWS * PARTS == 32, "a lane for every maximum and sum of the warp's rows");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch = lane % CH;
    // Row w (0 .. ROWS - 1) of the warp is row (w * 8 + warp) * PARTS + part of the item.  Its lanes w * PARTS + k fetch part
    // k's maximum and sum: a load of one address by the whole warp is as dear as 32 there.
    const float2 ml = ld_cluster_f32x2(pr_part_ml<D>(smem, ((lane / PARTS) * 8 + warp) * PARTS + part), lane % PARTS);
    float to = ml.x;
#pragma unroll
    for (int k = 1; k < PARTS; k <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, k));
    const float f = ml.y == 0.f ? 0.f : pr_ex2(ml.x - to);     // a part that saw nothing has weight 0
    float sum = f * ml.y;
#pragma unroll
    for (int k = 1; k < PARTS; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    const float w_part = sum != 0.f ? f / sum : 0.f;
    const float lse = sum == 0.f ? -INFINITY : (to + log2f(sum)) * 0.6931471805599453f;
#pragma unroll 1
    for (int x0 = 0; x0 < TURNS; x0 += BATCH) {
        float4 o[BATCH][PARTS];
        int64_t out[BATCH];        // the row in o, or none
#pragma unroll
        for (int y = 0; y < BATCH; ++y) {
            const int i = (((x0 + y) * AT_ONCE + lane / CH) * 8 + warp) * PARTS + part;
            const int t = i / PR_ROWS, row = i % PR_ROWS, tl = row / A.r, tok = tok0 + t * A.tq + tl;
            out[y] = tl < A.tq && tok < nq ? (qs + tok) * A.hq + g * A.r + row - tl * A.r : -1;
            if (out[y] < 0) continue;
#pragma unroll
            for (int k = 0; k < PARTS; ++k)
                o[y][k] = k == part ? *pr_part_row<D>(smem, i, ch) : ld_cluster_f32x4(pr_part_row<D>(smem, i, ch), k);
        }
#pragma unroll
        for (int y = 0; y < BATCH; ++y) {
            const int w = (x0 + y) * AT_ONCE + lane / CH;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                const float c = __shfl_sync(0xffffffffu, w_part, w * PARTS + k);
                if (c == 0.f) continue;        // its memory may hold anything
                acc.x += c * o[y][k].x;
                acc.y += c * o[y][k].y;
                acc.z += c * o[y][k].z;
                acc.w += c * o[y][k].w;
            }
            const float row_lse = __shfl_sync(0xffffffffu, lse, w * PARTS);
            if (out[y] < 0) continue;
            const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x, acc.y), b = __floats2bfloat162_rn(acc.z, acc.w);
            *reinterpret_cast<uint2*>(A.o + out[y] * D + 4 * ch) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
            if (ch == 0 && A.lse) A.lse[out[y]] = row_lse;
        }
    }
}

// SPLIT: a cluster of CTAs shares an item's keys and joins its parts.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(PR_THREADS, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PromptArgs A) {
    using P = PrShape<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PrShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int TU = 2 * A.tq;

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t ring = base + 2 * P::TILE;
    if (warp == 9 && lane == 0) {                 // the loading thread sets up the barriers: its first loads need no other
        tensor_map_prefetch(&map_q);
        tensor_map_prefetch(&map_k);
        tensor_map_prefetch(&map_v);
        for (int i = 0; i < P::STAGES; ++i) mbar_init(smem_u32(&sh.kv_full[i]), 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&sh.q_full[t]), 1);
            for (int i = 0; i < P::DEPTH; ++i) mbar_init(smem_u32(&sh.s_full[t][i]), 1);
            mbar_init(smem_u32(&sh.p_full[t][0]), 128);
            mbar_init(smem_u32(&sh.p_full[t][1]), 128);
            mbar_init(smem_u32(&sh.o_done[t]), 1);
            mbar_init(smem_u32(&sh.turn[t]), 1);
            mbar_init(smem_u32(&sh.drain[t]), 1);
        }
        mbar_init(smem_u32(&sh.v_tail), 1);
        sh.abort = sh.issued = sh.tail_open = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    grid_wait();
    if (blockIdx.x == 0 && A.status)           // bad offsets of any request, also of one that no item reaches
        for (int i = tid; i < A.batch; i += PR_THREADS) {
            const int64_t a = A.cu_q[i], e = A.cu_q[i + 1], c = A.cu_k[i], f = A.cu_k[i + 1];
            if (a < 0 || e < a || e > A.total_q || c < 0 || f < c || f > A.total_k) atomicOr(A.status, KVO_DEV_BAD_COUNT);
        }

    // Request b has ceil(nq / TU) items; its slots start at floor(cu_q[b] / TU) + b, which leaves room for them.
    const int parts = SPLIT ? (int)cluster_size() : 1, part = SPLIT ? (int)cluster_rank() : 0, item = blockIdx.x / parts;
    const int g = item % A.hkv, u = A.units - 1 - item / A.hkv;
    int64_t j0, qs, qe, ks, ke;
    if (A.batch <= 32) {                       // all offsets in one round of loads
        const bool have = lane < A.batch;
        const int a = have ? __ldg(A.cu_q + lane) : 0, e = have ? __ldg(A.cu_q + lane + 1) : 0;
        const int c = have ? __ldg(A.cu_k + lane) : 0, f = have ? __ldg(A.cu_k + lane + 1) : 0;
        const int64_t first = (int64_t)max(a, 0) / TU + lane;
        const int b = max(0, 31 - __clz((int)__ballot_sync(0xffffffffu, have && first <= u)));
        j0 = u - __shfl_sync(0xffffffffu, first, b);
        qs = __shfl_sync(0xffffffffu, a, b);
        qe = __shfl_sync(0xffffffffu, e, b);
        ks = __shfl_sync(0xffffffffu, c, b);
        ke = __shfl_sync(0xffffffffu, f, b);
        if (__any_sync(0xffffffffu, !offsets_ascend(a, e, A.total_q))) {
            const int at = find_served(a, e, A.batch, A.total_q, u, TU, 1);
            if (at < 0) return;
            qs = A.cu_q[at];
            qe = A.cu_q[at + 1];
            ks = A.cu_k[at];
            ke = A.cu_k[at + 1];
            j0 = u - ((int)qs / TU + at);
        }
    } else {
        auto first = [&](int i) { return (int64_t)max(__ldg(A.cu_q + i), 0) / TU + i; };
        const int b = warp_find(A.batch, u, first);
        j0 = u - first(b);
        qs = A.cu_q[b];
        qe = A.cu_q[b + 1];
        ks = A.cu_k[b];
        ke = A.cu_k[b + 1];
    }
    if (qs < 0 || qe < qs || qe > A.total_q || ks < 0 || ke < ks || ke > A.total_k) return;
    const int nq = (int)(qe - qs), nk = (int)(ke - ks);
    if (j0 < 0 || j0 * TU >= nq) return;
    const int tok0 = (int)j0 * TU;
    int n_t[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int have = min(max(nq - tok0 - t * A.tq, 0), A.tq);
        const int64_t see = A.causal ? min(max((int64_t)tok0 + t * A.tq + have + (nk - nq), (int64_t)0), (int64_t)nk) : nk;
        n_t[t] = have ? (int)((see + PR_KEYS - 1) / PR_KEYS) : 0;
    }
    int n = max(n_t[0], n_t[1]), first = 0;        // tiles of keys of this CTA, and the first of them
    if (SPLIT) {
        first = (int)((int64_t)n * part / parts);
        const int mine = (int)((int64_t)n * (part + 1) / parts) - first;
        n_t[0] = min(max(n_t[0] - first, 0), mine);
        n_t[1] = min(max(n_t[1] - first, 0), mine);
        n = max(n_t[0], n_t[1]);
    }
    const int key_first = first * PR_KEYS, nk_here = nk - key_first;
    ks += key_first;

    if (warp == 9 && lane == 0 && n > 0) {     // Q and the first keys
        mbar_expect_tx(smem_u32(&sh.kv_full[0]), P::TILE);
        for (int x = 0; x < D / 64 && A.skip != 0; ++x)
            tma_load_3d(ring + x * PR_BLOCK, &map_k, 64 * x, g, (int)ks, smem_u32(&sh.kv_full[0]));
        for (int t = 0; t < 2; ++t) {
            if (n_t[t] == 0) continue;         // a tile that sees no key: nothing reads its Q
            mbar_expect_tx(smem_u32(&sh.q_full[t]), (uint32_t)((D / 64) * 128 * A.r * A.tq));
            for (int x = 0; x < D / 64; ++x)
                tma_load_3d(base + t * P::TILE + x * PR_BLOCK, &map_q, 64 * x, g * A.r, (int)qs + tok0 + t * A.tq,
                            smem_u32(&sh.q_full[t]));
        }
    }
    __syncwarp();
    if (warp == 8) tmem_alloc(smem_u32(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp >= 8) {
        regs_dec<88>();
        if (warp == 9 && n > 0) {
            // ------------------------------------------------ loads
            int issued = 1;
            bool ok = true, tail_open = false;
            for (int i = 1; i < 2 * n; ++i) {
                const int st = i % P::STAGES, jj = i >> 1, key0 = jj * PR_KEYS;
                const bool is_v = i & 1;
                if (i >= P::STAGES) {
                    // K(jj - DEPTH)'s stage is free once both tiles' scores with it are there, V(jj - DEPTH)'s once the
                    // scores after it are, which were issued after its value product (n_t differ by one at most, so
                    // those exist).  Each of these barriers completes next with a tile that this loop loads later, so
                    // a parity says which phase is meant.
                    const int x = jj - P::DEPTH + is_v;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (x < n_t[t] && ok) ok = pr_wait(sh, A, sh.s_full[t][x % P::DEPTH], (x / P::DEPTH) & 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                const uint32_t dst = ring + st * P::TILE;
                // The last tile of a request runs into what lies behind it.  Its keys are masked as scores, but
                // a weight of zero does not silence a NaN or an infinity in V: those rows are cleared here.
                const bool tail = is_v && key0 + PR_KEYS > nk_here;
                const uint32_t bar = smem_u32(tail ? &sh.v_tail : &sh.kv_full[st]);
                if (lane == 0) {
                    mbar_expect_tx(bar, P::TILE);
                    for (int x = 0; x < D / 64 && i != A.skip; ++x)
                        tma_load_3d(dst + x * PR_BLOCK, is_v ? &map_v : &map_k, 64 * x, g, (int)ks + key0, bar);
                }
                if (tail) {
                    tail_open = true;
                    ok = pr_wait(sh, A, sh.v_tail, 0);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tail_open = false;
                    for (int x = 0; x < D / 64; ++x)
                        for (uint32_t a = (nk_here - key0) * 128 + lane * 16; a < PR_BLOCK; a += 512)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + x * PR_BLOCK + a), "r"(0) : "memory");
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.kv_full[st]));
                }
                issued = i + 1;
            }
            if (lane == 0) { sh.issued = issued; sh.tail_open = tail_open; }
        } else if ((warp & 1) == 0 && lane == 0 && n_t[(warp - 8) >> 1] > 0) {
            // ------------------------------------------------ matrix products of one tile
            // The tensor cores queue a few instructions only; with a thread of its own for each tile, one tile's
            // waits and commits (about 100 and 55 cycles) pass while the other's products run.  They take turns, so
            // that the tiles stay half a period apart: left alone both fall into step, and then the tensor cores
            // idle while both do their softmax.
            constexpr uint32_t ID_S = mma_desc(PR_ROWS, PR_KEYS, false), ID_O = mma_desc(PR_ROWS, D, true);
            const int t = (warp - 8) >> 1, n_mine = n_t[t], n_other = n_t[t ^ 1];
            const uint32_t S = sh.tmem + 128 * t, O = sh.tmem + 256 + D * t;
            const uint64_t q = smem_desc(base + t * P::TILE, 16), k0 = smem_desc(ring, 16), v0 = smem_desc(ring, PR_BLOCK);
            auto scores = [&](int stage, bool pass) {            // stage 2 (j % DEPTH) holds K(j)
                const uint64_t k = k0 + stage * (P::TILE >> 4);
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    if (e == D / 32 && pass) mbar_arrive(smem_u32(&sh.turn[t ^ 1]));     // queued work covers the hand-over
                    const int off = (e >> 2) * (PR_BLOCK >> 4) + (e & 3) * 2;
                    mma_ss(S, q + off, k + off, ID_S, e > 0);
                }
                tc_commit(smem_u32(&sh.s_full[t][stage >> 1]));
            };
            int ks = 0, vs = 1;                      // stages of K and V, and the parities of their next fill
            uint32_t kp = 0, vp = 0;
            bool ok = pr_wait(sh, A, sh.q_full[t], 0) && pr_wait(sh, A, sh.kv_full[0], 0);
            if (ok) scores(0, false);
            for (int j = 0; ok && j < n_mine; ++j) {
                ks += 2;
                if (ks >= P::STAGES) { ks -= P::STAGES; kp ^= 1; }
                if (!(ok = pr_wait(sh, A, sh.kv_full[vs], vp))) break;
                if (j + 1 < n_mine && !(ok = pr_wait(sh, A, sh.kv_full[ks], kp))) break;
                const uint64_t v = v0 + vs * (P::TILE >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {        // in two halves of the keys, each as its weights come
                    if (!ok || !(ok = pr_wait(sh, A, sh.p_full[t][h], j & 1))) break;
                    if (h == 0) {
                        const int k = t ? j : j - 1;             // the other tile's round before this one
                        if (k >= 0 && k < n_other && !(ok = pr_wait(sh, A, sh.turn[t], k & 1))) break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int e = 4 * h; e < 4 * h + 4; ++e)
                        mma_ts(O, S + 8 * e, v + e * (2048 >> 4), ID_O, j > 0 || e > 0);
                }
                if (!ok) break;
                // One commit for the scores stands for the value product before them as well.
                if (j + 1 < n_mine) {
                    scores(ks, true);
                } else {
                    tc_commit(smem_u32(&sh.o_done[t]));
                    mbar_arrive(smem_u32(&sh.turn[t ^ 1]));
                }
                vs += 2;
                if (vs >= P::STAGES) { vs -= P::STAGES; vp ^= 1; }
            }
            // nothing of this CTA may be in flight when it leaves
            tc_commit(smem_u32(&sh.drain[t]));
            if (!mbar_wait_bounded(smem_u32(&sh.drain[t]), 0, A.wait_ns)) {
                *(volatile int*)&sh.abort = 1;
                if (A.status) atomicOr(A.status, KVO_DEV_TIMEOUT);
            }
        }
        __syncwarp();
        if constexpr (SPLIT) { cluster_barrier(); cluster_barrier(); }     // as below
    } else {
        regs_inc<208>();
        const int t = warp >> 2, row = tid & 127;
        const int tl = row / A.r, head = row - tl * A.r;
        const int tok = tok0 + t * A.tq + tl;
        const bool real = tl < A.tq && tok < nq;
        int limit = 0;
        if (real) limit = A.causal ? (int)min(max((int64_t)tok + 1 + (nk - nq), (int64_t)0), (int64_t)nk) : nk;
        uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
        if (SPLIT) limit = max(limit - key_first, 0);
        pr_softmax<D, SPLIT>(sh, A, t, n_t[t], limit, real, (qs + tok) * A.hq + g * A.r + head, smem);
        if constexpr (SPLIT) {
            cluster_barrier();
            if (parts == 2) pr_join<D, 2>(A, smem, part, g, qs, nq, tok0);
            else if (parts == 4) pr_join<D, 4>(A, smem, part, g, qs, nq, tok0);
            else pr_join<D, 8>(A, smem, part, g, qs, nq, tok0);
            cluster_barrier();         // nobody leaves while its part is read
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_free(sh.tmem, 512);
    // Every warp has left its waits, so `abort` is final.  Where it is set somebody stopped before all loads had landed:
    // the thread that issued them stays until they have, and with it the CTA and its shared memory.
    if (warp == 9 && lane == 0 && sh.abort) {
        const int issued = sh.issued;
        for (int t = 0; t < 2; ++t)
            if (issued && n_t[t] > 0) mbar_wait_bounded(smem_u32(&sh.q_full[t]), 0, A.wait_ns);
        for (int i = max(0, issued - P::STAGES); i < issued; ++i)
            mbar_wait_bounded(smem_u32(&sh.kv_full[i % P::STAGES]), (i / P::STAGES) & 1, A.wait_ns);
        if (sh.tail_open) mbar_wait_bounded(smem_u32(&sh.v_tail), 0, A.wait_ns);
    }
}

template <int D, bool SPLIT>
cudaError_t prompt_attn_launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PromptArgs& A,
                               int parts, unsigned items, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    if (first_on_device(done)) {
        const cudaError_t e =
            cudaFuncSetAttribute(prompt_attn_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, PrShape<D>::SMEM);
        if (e != cudaSuccess) return e;
        mark_on_device(done);
    }
    return launch_dependent(prompt_attn_kernel<D, SPLIT>, dim3(items * parts), PR_THREADS, PrShape<D>::SMEM, s,
                            SPLIT ? parts : 0, q, k, v, A);
}

// How many CTAs share an item's keys: the number whose items end first by estimate.  The host knows means only: `items`
// items of `least` to `most` tiles of keys.  An item takes 1.36 us per tile and 6 us besides, 11 where parts are joined;
// 152 items run at once, or 76, 36 and 14 clusters of 2, 4 and 8 (as measured: larger clusters leave SMs idle).  The
// end is that of the longest item, or the mean time of the items in each place, the last round with the shortest.
// Measured in us, unsplit / split in 2 / 4 / 8, 32 and 8 heads of 128, tokens behind cached keys: 1 behind 8000 101 / 57
// / 32 / 19, 64 behind 2000 31 / 24 / 18 / 16, 512 behind 1500 29 / 23 / 34 / 65, 256 behind 32000 363 / 194 / 104 / 174,
// 1400 behind 32000 736 / 588 / 533 / 703; but 512 alone 12.3 / 14.3 / 25 / 58, 1024 behind 32000 374 / 389 / 417 / 523,
// 8192 alone 360 / 478 / 648 / 1143.  The estimate is within a fifth of these.
int prompt_attn_parts(int64_t items, int64_t least, int64_t most) {
    struct { int parts, fit; double us; } const choice[] = {{1, 152, 6.}, {2, 76, 11.}, {4, 36, 11.}, {8, 14, 11.}};
    const double lo = 1.36 * (double)least, hi = 1.36 * (double)most;
    int best = 1;
    double first = INFINITY;
    for (const auto& c : choice) {
        const double rounds = (double)items / c.fit;
        const double t = std::max(hi / c.parts + c.us, rounds * ((lo + hi) / 2 / c.parts + c.us) +
                                                           (ceil(rounds) - rounds) * (lo / c.parts + c.us));
        if (t < first) { first = t; best = c.parts; }
    }
    return best;
}

}  // namespace kvo

extern "C" kvo_status kvo_prompt_attn(const void* q, int64_t q_token_stride, const void* k, int64_t k_token_stride,
                                      const void* v, int64_t v_token_stride, const int32_t* cu_q, const int32_t* cu_k,
                                      int batch, int64_t total_q, int64_t total_k, int n_q_heads, int n_kv_heads,
                                      int head_dim, int causal, void* o, float* lse, int32_t* status,
                                      kvo_stream_t stream) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (batch < 0 || total_q < 0 || total_k < 0 || total_q > INT32_MAX || total_k > INT32_MAX)
        return bad("batch, total_q and total_k must be in 0..2^31 - 1");
    if (n_kv_heads < 1 || n_q_heads < n_kv_heads || n_q_heads % n_kv_heads)
        return bad("n_q_heads must be a multiple of n_kv_heads");
    const int r = n_q_heads / n_kv_heads;
    if (r > 16) return bad("n_q_heads / n_kv_heads must be <= 16");
    if (head_dim != 64 && head_dim != 128) return bad("head_dim must be 64 or 128");
    if (batch == 0 || total_q == 0) return KVO_OK;
    if (!q || !o || !cu_q || !cu_k || (total_k > 0 && (!k || !v))) return bad("null pointer argument");
    for (const void* p : {q, k, v, (const void*)o})
        if ((uintptr_t)p % 16) return bad("q, k, v and o must be 16-byte aligned");
    if (q_token_stride % 8 || k_token_stride % 8 || v_token_stride % 8) return bad("strides must be multiples of 8 elements");
    if (q_token_stride < (int64_t)n_q_heads * head_dim || k_token_stride < (int64_t)n_kv_heads * head_dim ||
        v_token_stride < (int64_t)n_kv_heads * head_dim)
        return bad("token strides must cover the heads");
    if (q_token_stride > (1ll << 38) || k_token_stride > (1ll << 38) || v_token_stride > (1ll << 38))
        return bad("token strides must be below 2^38 elements");
    const int64_t o_bytes = rows_bytes(total_q, (int64_t)n_q_heads * head_dim, (int64_t)n_q_heads * head_dim);
    if (ranges_meet(o, o_bytes, q, rows_bytes(total_q, q_token_stride, (int64_t)n_q_heads * head_dim)) ||
        ranges_meet(o, o_bytes, k, rows_bytes(total_k, k_token_stride, (int64_t)n_kv_heads * head_dim)) ||
        ranges_meet(o, o_bytes, v, rows_bytes(total_k, v_token_stride, (int64_t)n_kv_heads * head_dim)))
        return bad("o must not overlap q, k or v");
    const Bytes to_o{o, o_bytes}, to_lse{lse, 4 * total_q * n_q_heads};
    const int64_t cu_bytes = 4 * ((int64_t)batch + 1);
    if (meets_any(to_o, {to_lse, {cu_q, cu_bytes}, {cu_k, cu_bytes}}) ||
        meets_any(to_lse, {{q, rows_bytes(total_q, q_token_stride, (int64_t)n_q_heads * head_dim)},
                           {k, rows_bytes(total_k, k_token_stride, (int64_t)n_kv_heads * head_dim)},
                           {v, rows_bytes(total_k, v_token_stride, (int64_t)n_kv_heads * head_dim)},
                           {cu_q, cu_bytes}, {cu_k, cu_bytes}}))
        return bad("o and lse must be apart from each other and from all that the call reads");
    PromptArgs A{};
    A.cu_q = cu_q;
    A.cu_k = cu_k;
    A.o = (uint16_t*)o;
    A.lse = lse;
    A.status = status;
    A.total_q = total_q;
    A.total_k = total_k;
    A.batch = batch;
    A.hq = n_q_heads;
    A.hkv = n_kv_heads;
    A.r = r;
    A.tq = PR_ROWS / r;
    A.causal = causal ? 1 : 0;
    A.scale_log2 = (float)(1.4426950408889634 / sqrt((double)head_dim));
    A.skip = call_wait.skip;
    A.wait_ns = call_wait.limit_ns;
    const int64_t units = total_q / (2 * A.tq) + batch, ctas = units * n_kv_heads;
    if (ctas > INT32_MAX) return bad("too many tokens");
    A.units = (int)units;
    CUtensorMap mq, mk, mv;
    const uint64_t sq[3] = {(uint64_t)head_dim, (uint64_t)n_q_heads, (uint64_t)total_q};
    const uint64_t sk[3] = {(uint64_t)head_dim, (uint64_t)n_kv_heads, (uint64_t)std::max<int64_t>(total_k, 1)};
    const uint64_t tq[2] = {(uint64_t)head_dim * 2, (uint64_t)q_token_stride * 2};
    const uint64_t tk[2] = {(uint64_t)head_dim * 2, (uint64_t)k_token_stride * 2};
    const uint64_t tv[2] = {(uint64_t)head_dim * 2, (uint64_t)v_token_stride * 2};
    const uint32_t bq[3] = {64, (uint32_t)r, (uint32_t)A.tq}, bk[3] = {64, 1, PR_KEYS};
    // without keys the maps of k and v are never used: q stands in for a null pointer
    if (!tensor_map(&mq, q, 2, 3, sq, tq, bq) || !tensor_map(&mk, total_k ? k : q, 2, 3, sk, tk, bk) ||
        !tensor_map(&mv, total_k ? v : q, 2, 3, sk, tv, bk)) {
        set_last_error("cuTensorMapEncodeTiled failed for q, k or v");
        return KVO_ERR_CUDA;
    }
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t tu = 2 * A.tq, items = std::max((total_q + tu - 1) / tu, std::min<int64_t>(batch, total_q)) * n_kv_heads;
    const int64_t keys = total_k / batch, unseen = causal ? std::min(total_q / batch, keys) : 0;    // by the first token
    const int parts = prompt_attn_parts(items, (keys - unseen + PR_KEYS - 1) / PR_KEYS, (keys + PR_KEYS - 1) / PR_KEYS);
    if (ctas * parts > INT32_MAX) return bad("too many tokens");
    cudaError_t e;
#define KVO_PROMPT(D_) (parts > 1 ? prompt_attn_launch<D_, true>(mq, mk, mv, A, parts, (unsigned)ctas, s) : prompt_attn_launch<D_, false>(mq, mk, mv, A, 1, (unsigned)ctas, s))
    e = head_dim == 128 ? KVO_PROMPT(128) : KVO_PROMPT(64);
#undef KVO_PROMPT
    if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    return KVO_OK;
}
