// The paged device cache: layout, checks and small device helpers shared by the
// append and the attention that reads it.
//
// Page p of KV head h holds page_size rows of head_dim values, contiguous:
// [n_pages][Hkv][page_size][head_dim], bf16 or e4m3.  In e4m3 a value is
// code * scale[p][h].  Token t of request b lives in row t % page_size of page
// table[b][t / page_size].
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include <initializer_list>

#include "kvo_internal.cuh"

namespace kvo {

constexpr float E4M3_MAX = 448.f;

// Two floats -> two e4m3 codes (lo in the low byte), to nearest even, +-448 beyond; NaN stays NaN.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes -> f16x2 (exact: every e4m3 value is an f16 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// Smallest power of two s >= 2^-100 with amax <= 448 s, amax finite: with
// amax = m 2^e, m in [1, 2), that is 2^(e - 8) up to m = 1.75 and 2^(e - 7) above.
// A power of two makes code * s, and a page's move to a larger scale, exact
// above the subnormal codes; it costs no precision, since a float format's
// relative step is the same at every binade.
__device__ __forceinline__ float e4m3_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

// The last i in [0, n) with first(i) <= key, for a non-decreasing `first` with
// first(0) <= key; called by a whole warp, 32 probes a round.  Terminates (with
// some index in range) whatever `first` returns.
template <typename F>
__device__ __forceinline__ int warp_find(int n, int64_t key, F first) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const bool le = at < n && first(lo + at) <= key;
        const int k = max(0, 31 - __clz((int)__ballot_sync(0xffffffffu, le)));
        lo += k * step;
        n = max(1, min(step, n - k * step));
    }
    return lo;
}

// Packed requests: request i's rows are cu[i] .. cu[i + 1] - 1 of `total`.  It is served where its offsets ascend within
// 0..total and it begins at or behind the end of every earlier request of which that is true, so no row belongs to two.
// Request i's work starts at slot cu[i] / rows + extra * i and has n / rows + extra slots: those of served requests do not
// meet, and where all offsets ascend the last request that starts at or before a slot holds it.  A warp sees at a glance
// whether they do for up to 32 requests (a lane each); calls of more take them as they are: for each CTA to look at all
// of them cost 4 % of a call of 33 requests and 28 % of one of 4000.
__device__ __forceinline__ bool offsets_ascend(int a, int e, int64_t total) { return a >= 0 && e >= a && e <= total; }

// Whole warp, up to 32 requests, lane i with offsets a and e of request i: the served request that holds a slot, or -1,
// whatever the offsets are.
static __device__ __noinline__ int find_served(int a, int e, int batch, int64_t total, int slot, int rows, int extra) {
    const int lane = threadIdx.x & 31;
    const bool own = lane < batch && offsets_ascend(a, e, total);
    int end = own ? e : 0;         // the end of the requests up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end = max(end, x);
    }
    const int before = __shfl_up_sync(0xffffffffu, end, 1), first = max(a, 0) / rows + extra * lane;
    return __ffs((int)__ballot_sync(0xffffffffu, own && (lane == 0 || a >= before) && slot >= first && slot < first + (e - a) / rows + extra)) - 1;
}

// Host: whether two byte ranges share a byte.
inline bool ranges_meet(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}
// Host: whether a byte range shares a byte with any of some others (null pointers: none).
struct Bytes {
    const void* at;
    int64_t n;
};
inline bool meets_any(const Bytes& x, std::initializer_list<Bytes> others) {
    for (const Bytes& y : others)
        if (x.at && y.at && ranges_meet(x.at, x.n, y.at, y.n)) return true;
    return false;
}
// Host: bytes of a cache's pages of K (and of V), and of their scales.
inline int64_t page_bytes(const kvo_paged_cache* c) {
    return (int64_t)c->n_pages * c->n_kv_heads * c->page_size * c->head_dim * (c->format == KVO_PAGES_E4M3 ? 1 : 2);
}
inline int64_t scale_bytes(const kvo_paged_cache* c) { return c->format == KVO_PAGES_E4M3 ? 4ll * c->n_pages * c->n_kv_heads : 0; }
// Host: bytes from the first to the last of `n` bf16 rows of `len` values, `stride` apart.
inline int64_t rows_bytes(int64_t n, int64_t stride, int64_t len) { return n > 0 ? 2 * ((n - 1) * stride + len) : 0; }

// Host: a message for a cache descriptor that no call may use, or NULL.
inline const char* paged_cache_error(const kvo_paged_cache* c) {
    if (!c) return "null cache";
    if (c->batch < 0 || c->n_kv_heads < 1) return "need batch >= 0 and n_kv_heads >= 1";
    if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return "page_size must be 16, 32, 64 or 128";
    if (c->n_pages < 1 || c->max_pages < 1) return "need n_pages >= 1 and max_pages >= 1";
    if ((int64_t)c->max_pages * c->page_size >= (1 << 30)) return "max_pages * page_size must fit in 30 bits";
    if ((int64_t)c->n_pages * c->n_kv_heads * c->page_size > INT32_MAX)
        return "n_pages * n_kv_heads * page_size must fit in 31 bits";
    if ((int64_t)c->batch * c->n_kv_heads > (1 << 20)) return "batch * n_kv_heads must be <= 2^20";
    if (c->format != KVO_PAGES_BF16 && c->format != KVO_PAGES_E4M3) return "format must be KVO_PAGES_BF16 or KVO_PAGES_E4M3";
    if (!c->k_pages || !c->v_pages || (!c->table && c->batch > 0)) return "null pages or table";
    if ((uintptr_t)c->k_pages % 16 || (uintptr_t)c->v_pages % 16) return "pages must be 16-byte aligned";
    if (c->format == KVO_PAGES_E4M3 && (!c->k_scale || !c->v_scale)) return "e4m3 pages need k_scale and v_scale";
    return nullptr;
}

}  // namespace kvo
