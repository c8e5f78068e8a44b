// kvo_paged_append: new keys and values into a paged cache, keys (and the
// queries beside them) rotated on the way.
//
// A key is rotated in fp32 and rounded once to bf16: that value goes to k_out
// and to bf16 pages, and it is what e4m3 pages quantise.  The one rounding
// step before the quantisation (2^-9 relative against e4m3's 2^-4) makes the
// prompt's own attention and the cache agree on what the key is.
//
// Prompts: one CTA owns one page that the call touches, of one to eight KV heads,
// so a page's scale needs no atomics: it holds the page's new rows in registers,
// takes their largest magnitude, settles the scale, moves rows of earlier calls
// to it when it grew, and writes codes.  q is rotated by further CTAs of the same
// launch, behind those of the pages (a second kernel that starts beside the last
// pages took 70.3 us for 64.1 with pages of 16 rows, 65.4 for 66.0 with 64, 6.1 for
// 4.8 at 500 tokens in pages of 16, and 4 us more of the host).  16391 tokens, 32 and 8
// heads of 128 with k_out, e4m3 pages of 64: 65.5 us, 6.15 TB/s (0.90 of a measured copy).
//
// One token per request: a warp owns one (token, head), of K and V or of q; each
// lane turns D / 64 pairs, so the angles take one or two sincos in a row.  Bound by a
// chain of dependent loads (start, page, old scale): 64 tokens, 32 and 8 heads of 128,
// e4m3, in 3.1 us.
//
#include <stdio.h>

#include <algorithm>

#include "launch.cuh"
#include "paged.cuh"
#include "rope.cuh"

namespace kvo {

constexpr int APP_THREADS = 256;              // of a CTA, unless pages are small or very large

struct AppendArgs {
    uint8_t* pages[2];            // K, V
    float* scale[2];
    const int32_t* table;
    const uint16_t* x[2];         // k, v
    int64_t x_tok[2];
    const int32_t* cu;            // [batch + 1] or NULL: one token each
    const int32_t* start;         // [batch]
    const uint16_t* q;
    uint16_t* q_out;
    uint16_t* k_out;
    int32_t* status;
    int64_t tokens, q_tok;
    int batch, hkv, hq, page, n_pages, max_pages;
    int runs, run;                // a CTA of pages takes `run` KV heads, `runs` CTAs a page
    int q_per, q_blocks;          // query heads per thread; CTAs for a run of so many
    int page_ctas;                // CTAs of pages; those after them rotate q
    RopeArgs R;
};

__device__ __forceinline__ void set_status(int32_t* status, int bits) {
    if (status && bits) atomicOr(status, bits);
}

// Request b's token range; false (with a status bit) when the caller's offsets
// leave [0, tokens] or the start is negative.
__device__ __forceinline__ bool request_range(const AppendArgs& A, int b, int64_t& t0, int64_t& n, int& start) {
    t0 = A.cu[b];
    n = (int64_t)A.cu[b + 1] - t0;
    start = A.start[b];
    return t0 >= 0 && n >= 0 && t0 + n <= A.tokens && start >= 0;
}

// Moves `words` 16-byte words of codes to another scale: thread i of n.
__device__ __forceinline__ void rescale_rows(uint8_t* codes, int words, float ratio, int i, int n) {
    uint4* row = reinterpret_cast<uint4*>(codes);
    for (int w = i; w < words; w += n) {
        uint4 v = row[w];
        uint16_t* cv = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t hh = e4m3x2_to_f16x2(cv[e]);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh));
            cv[e] = f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
        }
        row[w] = v;
    }
}

// Which request and which of its touched pages unit u is.  Request b has at most floor(n / page) + 2 of them, so its
// units start at floor(cu[b] / page) + 2 b: every request finds its own without a scan.  By a whole warp.
struct AppendUnit {
    int b, j, start;
    int64_t t0, n;
    bool ok;
};
__device__ __forceinline__ AppendUnit append_unit(const AppendArgs& A, int u) {
    AppendUnit U;
    if (A.batch <= 32) {           // all offsets and starts in one round of loads
        const int lane = threadIdx.x & 31;
        const bool have = lane < A.batch;
        const int c0 = have ? __ldg(A.cu + lane) : 0, c1 = have ? __ldg(A.cu + lane + 1) : 0;
        const int st = have ? __ldg(A.start + lane) : 0;
        const int64_t first = (int64_t)max(c0, 0) / A.page + 2 * (int64_t)lane;
        U.b = max(0, 31 - __clz((int)__ballot_sync(0xffffffffu, have && first <= u)));
        U.j = u - (int)__shfl_sync(0xffffffffu, first, U.b);
        U.t0 = __shfl_sync(0xffffffffu, c0, U.b);
        U.n = (int64_t)__shfl_sync(0xffffffffu, c1, U.b) - U.t0;
        U.start = __shfl_sync(0xffffffffu, st, U.b);
        U.ok = U.t0 >= 0 && U.n >= 0 && U.t0 + U.n <= A.tokens && U.start >= 0;
        if (__any_sync(0xffffffffu, !offsets_ascend(c0, c1, A.tokens))) {
            U.b = find_served(c0, c1, A.batch, A.tokens, u, A.page, 2);
            U.ok = U.b >= 0 && request_range(A, U.b, U.t0, U.n, U.start);
            if (U.ok) U.j = u - ((int)U.t0 / A.page + 2 * U.b);
        }
    } else {
        auto first = [&](int i) { return (int64_t)max(__ldg(A.cu + i), 0) / A.page + 2 * (int64_t)i; };
        U.b = warp_find(A.batch, u, first);
        U.j = u - (int)first(U.b);
        U.ok = request_range(A, U.b, U.t0, U.n, U.start);
    }
    return U;
}

// Bad offsets of any request, also of one that no unit reaches; by one CTA of the launch.
__device__ __forceinline__ void append_check(const AppendArgs& A) {
    for (int i = threadIdx.x; i < A.batch; i += blockDim.x) {
        int64_t t0, n;
        int start;
        if (!request_range(A, i, t0, n, start)) set_status(A.status, KVO_DEV_BAD_COUNT);
    }
}

// Largest magnitude of 8 bf16 values as bit patterns (a bf16 magnitude orders as its 15 bits), two lanes a word.
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, const uint4& v) {
    m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}
constexpr uint32_t BF16_INF = 0x7F80u;
// The same over the finite values only.
__device__ __forceinline__ uint32_t abs_max2_finite(uint32_t m, const uint4& v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t w = (&v.x)[e >> 1], x = ((e & 1) ? w >> 16 : w) & 0x7FFFu;
        if (x < BF16_INF) m = max(m, x);
    }
    return m;
}
// Eight bf16 values to eight codes of scale 1 / inv.  FINITE: none is an infinity (cvt would saturate it to 448 s;
// NaN keeps it visible).
template <bool FINITE>
__device__ __forceinline__ uint2 quantise8(const uint4& v, float inv) {
    uint32_t codes[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = (&v.x)[e];
        float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
        if (!FINITE) {
            lo = fabsf(lo) < INFINITY ? lo : NAN;
            hi = fabsf(hi) < INFINITY ? hi : NAN;
        }
        const uint32_t two = f32x2_to_e4m3x2(lo * inv, hi * inv);
        codes[e >> 1] = (e & 1) ? codes[e >> 1] | (two << 16) : two;
    }
    return make_uint2(codes[0], codes[1]);
}

// One thread, up to 32 requests: the served one that holds a row, or -1, whatever the offsets are.
static __device__ __noinline__ int find_served_row(const int32_t* cu, int batch, int64_t total, int64_t row) {
    int before = 0;
    for (int i = 0; i < batch; ++i) {
        const int a = __ldg(cu + i), e = __ldg(cu + i + 1);
        if (!offsets_ascend(a, e, total)) continue;
        if (a >= before && row >= a && row < e) return i;
        before = max(before, e);
    }
    return -1;
}

// Rotates packed q: CTA `block` of them takes (token, unit) pairs of a run of q_per heads.
template <int D>
__device__ __forceinline__ void append_q(const AppendArgs& A, int block) {
    constexpr int UNITS = D / 16;
    const int run = block / A.q_blocks;
    const int64_t k = (int64_t)(block - run * A.q_blocks) * blockDim.x + threadIdx.x, t = k / UNITS;
    const int mine = threadIdx.x & 31;
    const bool look = A.batch <= 32 && mine < A.batch;
    const int c0 = look ? __ldg(A.cu + mine) : 0, c1 = look ? __ldg(A.cu + mine + 1) : 0;
    const int u = (int)(k - t * UNITS);
    int lo = 0, hi = A.batch;                                  // the last b with cu[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (__ldg(A.cu + mid) <= t) lo = mid; else hi = mid;
    }
    int64_t t0, n;
    int start;
    bool ok = request_range(A, lo, t0, n, start);
    if (__any_sync(0xffffffffu, !offsets_ascend(c0, c1, A.tokens))) {
        lo = find_served_row(A.cu, A.batch, A.tokens, t);
        ok = lo >= 0 && request_range(A, lo, t0, n, start);
    }
    if (k < A.tokens * UNITS && ok && t >= t0 && t < t0 + n) {
        const int h0 = run * A.q_per, h1 = min(A.hq, h0 + A.q_per);
        rope_heads(A.R, D, A.q + t * A.q_tok, D, A.q_out + t * A.hq * D, D, u, (int)(start + (t - t0)), h0, h1);
    }
}

// A page's heads, by at most MAXT threads with MAXU units each.  AHEAD: the next head's rows are fetched while this
// one's are worked on, and the angles make room for them in shared memory, [4 MAXU][MAXT] (dynamic).
template <int D, bool FP8, int MAXU, int MAXT, bool AHEAD>
__global__ void __launch_bounds__(MAXT) append_pages_kernel(const __grid_constant__ AppendArgs A) {
    constexpr int UNITS = D / 16;                       // 16-value units of a row
    const int block = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, NT = blockDim.x;
    const int u = block / A.runs, h0 = (block - u * A.runs) * A.run, h1 = min(A.hkv, h0 + A.run);
    __shared__ uint32_t red[2][2][MAXT / 32];           // by the head's parity: one barrier a head
    extern __shared__ float4 angles[];
    auto angle = [&](int i) -> float4& { return angles[i * MAXT + tid]; };

    grid_wait();
    if (block == 0 && A.status) append_check(A);
    if (block >= A.page_ctas) {
        append_q<D>(A, block - A.page_ctas);
        return;
    }
    const AppendUnit U = append_unit(A, u);
    if (!U.ok) return;
    const int start = U.start;
    const int64_t at = start / A.page + (int64_t)U.j;       // logical page
    const int64_t pos0 = max((int64_t)start, at * A.page), pos1 = min(start + U.n, (at + 1) * A.page);
    if (pos0 >= pos1) return;
    if (at >= A.max_pages) {
        if (tid == 0 && h0 == 0) set_status(A.status, KVO_DEV_BAD_COUNT);
        return;
    }
    const int p = A.table[(int64_t)U.b * A.max_pages + at];
    const int row0 = (int)(pos0 - at * A.page), rows = (int)(pos1 - pos0);
    const int64_t tok0 = U.t0 + (pos0 - start);

    // this thread's units: row, first values of the two chunks, and the angles, shared by the heads
    int row[MAXU], ca[MAXU], cb[MAXU];
    float c[MAXU][8], s[MAXU][8];
    bool rot[MAXU];
    uint4 xa[2][MAXU], xb[2][MAXU], na[2][MAXU], nb[2][MAXU];
    auto load = [&](int h, uint4 (&xa)[2][MAXU], uint4 (&xb)[2][MAXU]) {
#pragma unroll
        for (int i = 0; i < MAXU; ++i)
            if (row[i] < rows) {
                const uint16_t* k = A.x[0] + (tok0 + row[i]) * A.x_tok[0] + (int64_t)h * D;
                const uint16_t* v = A.x[1] + (tok0 + row[i]) * A.x_tok[1] + (int64_t)h * D;
                xa[0][i] = *reinterpret_cast<const uint4*>(k + ca[i]);
                xb[0][i] = *reinterpret_cast<const uint4*>(k + cb[i]);
                xa[1][i] = *reinterpret_cast<const uint4*>(v + ca[i]);
                xb[1][i] = *reinterpret_cast<const uint4*>(v + cb[i]);
            }
    };
#pragma unroll
    for (int i = 0; i < MAXU; ++i) {
        const int w = tid + i * NT;
        row[i] = w / UNITS;
        rope_chunks(A.R, D, w % UNITS, ca[i], cb[i]);
    }
    load(h0, xa, xb);
    if (p < 0 || p >= A.n_pages) {                          // checked while the rows are on their way
        if (tid == 0 && h0 == 0) set_status(A.status, KVO_DEV_BAD_BLOCK_ID);
        return;
    }
#pragma unroll
    for (int i = 0; i < MAXU; ++i)
        rot[i] = row[i] < rows && rope_unit(A.R, (tid + i * NT) % UNITS, (int)(pos0 + row[i]), c[i], s[i]);

    if (AHEAD) {
#pragma unroll
        for (int i = 0; i < MAXU; ++i)
            if (rot[i]) {
                angle(4 * i) = make_float4(c[i][0], c[i][1], c[i][2], c[i][3]);
                angle(4 * i + 1) = make_float4(c[i][4], c[i][5], c[i][6], c[i][7]);
                angle(4 * i + 2) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
                angle(4 * i + 3) = make_float4(s[i][4], s[i][5], s[i][6], s[i][7]);
            }
    }
    for (int h = h0; h < h1; ++h) {
        if (AHEAD) {
            if (h > h0) {
#pragma unroll
                for (int i = 0; i < MAXU; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) { xa[x][i] = na[x][i]; xb[x][i] = nb[x][i]; }
            }
            if (h + 1 < h1) load(h + 1, na, nb);
        } else if (h > h0) {
            load(h, xa, xb);
        }
        const int64_t slot = (int64_t)p * A.hkv + h;
        float old[2] = {0.f, 0.f};
        if (FP8 && row0 > 0) { old[0] = A.scale[0][slot]; old[1] = A.scale[1][slot]; }
        uint32_t top[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < MAXU; ++i) {
            if (row[i] >= rows) continue;
            if (rot[i]) {
                if (AHEAD) {       // the thread's own words
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 vc = angle(4 * i + e), vs = angle(4 * i + 2 + e);
                        c[i][4 * e] = vc.x; c[i][4 * e + 1] = vc.y; c[i][4 * e + 2] = vc.z; c[i][4 * e + 3] = vc.w;
                        s[i][4 * e] = vs.x; s[i][4 * e + 1] = vs.y; s[i][4 * e + 2] = vs.z; s[i][4 * e + 3] = vs.w;
                    }
                }
                rope_rotate(A.R.interleaved, c[i], s[i], xa[0][i], xb[0][i]);
            }
            if (A.k_out) {
                uint16_t* o = A.k_out + ((tok0 + row[i]) * A.hkv + h) * D;
                *reinterpret_cast<uint4*>(o + ca[i]) = xa[0][i];
                *reinterpret_cast<uint4*>(o + cb[i]) = xb[0][i];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (FP8) {
                    top[x] = abs_max2(abs_max2(top[x], xa[x][i]), xb[x][i]);
                } else {
                    uint16_t* o = reinterpret_cast<uint16_t*>(A.pages[x]) + (slot * A.page + row0 + row[i]) * D;
                    *reinterpret_cast<uint4*>(o + ca[i]) = xa[x][i];
                    *reinterpret_cast<uint4*>(o + cb[i]) = xb[x][i];
                }
            }
        }
        if (!FP8) continue;
        auto block_max = [&](int x, uint32_t m) {           // contains the barrier after the second call
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) red[h & 1][x][warp] = m;
        };
        auto read_max = [&](int x) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < MAXT / 32; ++i)
                if (i < NT / 32) m = max(m, red[h & 1][x][i]);
            return m;
        };
#pragma unroll
        for (int x = 0; x < 2; ++x) block_max(x, max(top[x] & 0xFFFFu, top[x] >> 16));
        __syncthreads();
        uint32_t m[2] = {read_max(0), read_max(1)};
        const bool finite = m[0] < BF16_INF && m[1] < BF16_INF;
        if (!finite) {                                      // rare, the same for the whole CTA: leave out what is not finite
            __syncthreads();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t t = 0;
#pragma unroll
                for (int i = 0; i < MAXU; ++i)
                    if (row[i] < rows) t = abs_max2_finite(abs_max2_finite(t, xa[x][i]), xb[x][i]);
                block_max(x, t);
            }
            __syncthreads();
            m[0] = read_max(0);
            m[1] = read_max(1);
        }
        float inv[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float sc = e4m3_scale(__uint_as_float(m[x] << 16));
            if (row0 > 0) {                                 // rows of earlier calls: the scale never shrinks
                sc = fmaxf(sc, old[x]);
                if (sc != old[x]) rescale_rows(A.pages[x] + slot * A.page * D, row0 * UNITS, old[x] / sc, tid, NT);
            }
            if (tid == 0) A.scale[x][slot] = sc;            // every thread read the old one before the barrier
            inv[x] = 1.f / sc;
        }
#pragma unroll
        for (int i = 0; i < MAXU; ++i) {
            if (row[i] >= rows) continue;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint8_t* o = A.pages[x] + (slot * A.page + row0 + row[i]) * D;
                *reinterpret_cast<uint2*>(o + ca[i]) = finite ? quantise8<true>(xa[x][i], inv[x]) : quantise8<false>(xa[x][i], inv[x]);
                *reinterpret_cast<uint2*>(o + cb[i]) = finite ? quantise8<true>(xb[x][i], inv[x]) : quantise8<false>(xb[x][i], inv[x]);
            }
        }
    }
}

constexpr int STEP_WARPS = 4;

// One token per request: warp (b, h) appends K and V of KV head h, or rotates query head h - Hkv.
// Lane i holds slots i * N .. i * N + N - 1 of the head's D / 2: slot s is pair s of the rotated part, or values
// 2 s, 2 s + 1 of the rest.
template <int D, bool FP8>
__global__ void __launch_bounds__(STEP_WARPS * 32) append_step_kernel(const __grid_constant__ AppendArgs A) {
    constexpr int N = D / 64;
    const int lane = threadIdx.x & 31, heads = A.hkv + (A.q ? A.hq : 0);
    const int64_t w = (int64_t)blockIdx.x * STEP_WARPS + (threadIdx.x >> 5);
    grid_wait();
    if (w >= (int64_t)A.batch * heads) return;
    const int b = (int)(w / heads), h = (int)(w - (int64_t)b * heads);
    const bool is_q = h >= A.hkv;
    const uint16_t* x = is_q ? A.q + b * A.q_tok + (h - A.hkv) * D : A.x[0] + b * A.x_tok[0] + h * D;
    const int start = __ldg(A.start + b);
    const int s0 = lane * N;
    const bool rot = 2 * s0 < A.R.rot_dim, split = rot && !A.R.interleaved;
    const int ca = split ? s0 : 2 * s0, cb = split ? s0 + A.R.rot_dim / 2 : 2 * s0 + N;   // the two groups of N values
    uint16_t xa[N], xb[N];
    uint16_t v[2 * N];
    if constexpr (N == 2) {
        const uint32_t a = *reinterpret_cast<const uint32_t*>(x + ca), c = *reinterpret_cast<const uint32_t*>(x + cb);
        xa[0] = (uint16_t)a; xa[1] = (uint16_t)(a >> 16); xb[0] = (uint16_t)c; xb[1] = (uint16_t)(c >> 16);
    } else {
        xa[0] = x[ca]; xb[0] = x[cb];
    }
    if (!is_q) {
        const uint16_t* y = A.x[1] + b * A.x_tok[1] + h * D + 2 * s0;
        if constexpr (N == 2) {
            const uint2 a = *reinterpret_cast<const uint2*>(y);
            v[0] = (uint16_t)a.x; v[1] = (uint16_t)(a.x >> 16); v[2] = (uint16_t)a.y; v[3] = (uint16_t)(a.y >> 16);
        } else {
            const uint32_t a = *reinterpret_cast<const uint32_t*>(y);
            v[0] = (uint16_t)a; v[1] = (uint16_t)(a >> 16);
        }
    }
    unsigned long long freq[N];
#pragma unroll
    for (int i = 0; i < N; ++i) freq[i] = rot ? __ldg(A.R.freq + s0 + i) : 0ull;
    // The page (and its scale) are fetched before the angles are computed.
    const int at = start / A.page, row0 = start - at * A.page;
    int p = -1;
    bool bad = start < 0;
    if (!is_q && !bad) {
        if (at >= A.max_pages) bad = true; else p = __ldg(A.table + (int64_t)b * A.max_pages + at);
    }
    const bool good = !is_q && p >= 0 && p < A.n_pages;
    float old[2] = {0.f, 0.f};
    if (FP8 && good && row0 > 0) {
        old[0] = A.scale[0][(int64_t)p * A.hkv + h];
        old[1] = A.scale[1][(int64_t)p * A.hkv + h];
    }
    if (rot) {
        float f[2 * N];            // xa, xb as they come: pair i is (xa[i], xb[i]), or neighbours where interleaved
#pragma unroll
        for (int i = 0; i < N; ++i) { f[i] = __uint_as_float((uint32_t)xa[i] << 16); f[N + i] = __uint_as_float((uint32_t)xb[i] << 16); }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float c, s;
            rope_sincos(start, freq[i], A.R.amp, c, s);
            const float u0 = A.R.interleaved ? f[2 * i] : f[i], v0 = A.R.interleaved ? f[2 * i + 1] : f[N + i];
            const float nu = u0 * c - v0 * s, nv = u0 * s + v0 * c;
            if (A.R.interleaved) { f[2 * i] = nu; f[2 * i + 1] = nv; } else { f[i] = nu; f[N + i] = nv; }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            xa[i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
            xb[i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[N + i]));
        }
    }
    auto store = [&](uint16_t* o) {      // the rotated row of D values
        if constexpr (N == 2) {
            *reinterpret_cast<uint32_t*>(o + ca) = (uint32_t)xa[0] | (uint32_t)xa[1] << 16;
            *reinterpret_cast<uint32_t*>(o + cb) = (uint32_t)xb[0] | (uint32_t)xb[1] << 16;
        } else {
            o[ca] = xa[0]; o[cb] = xb[0];
        }
    };
    if (is_q) {
        if (!bad) store(A.q_out + ((int64_t)b * A.hq + h - A.hkv) * D);
        return;
    }
    if (!good) {
        if (lane == 0 && h == 0) set_status(A.status, bad ? KVO_DEV_BAD_COUNT : KVO_DEV_BAD_BLOCK_ID);
        return;
    }
    if (A.k_out) store(A.k_out + ((int64_t)b * A.hkv + h) * D);
    const int64_t base = (((int64_t)p * A.hkv + h) * A.page + row0) * D;
    if constexpr (!FP8) {
        store(reinterpret_cast<uint16_t*>(A.pages[0]) + base);
        uint16_t* o = reinterpret_cast<uint16_t*>(A.pages[1]) + base + 2 * s0;
        if constexpr (N == 2)
            *reinterpret_cast<uint2*>(o) = make_uint2((uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16);
        else
            *reinterpret_cast<uint32_t*>(o) = (uint32_t)v[0] | (uint32_t)v[1] << 16;
    } else {
        float f[2][2 * N], top[2] = {0.f, 0.f}, inv[2];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            f[0][i] = __uint_as_float((uint32_t)xa[i] << 16);
            f[0][N + i] = __uint_as_float((uint32_t)xb[i] << 16);
            f[1][2 * i] = __uint_as_float((uint32_t)v[2 * i] << 16);
            f[1][2 * i + 1] = __uint_as_float((uint32_t)v[2 * i + 1] << 16);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int i = 0; i < 2 * N; ++i)
                if (fabsf(f[y][i]) < INFINITY) top[y] = fmaxf(top[y], fabsf(f[y][i]));
#pragma unroll
            for (int o = 16; o; o >>= 1) top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], o));
            float s = e4m3_scale(top[y]);
            if (row0 > 0) {
                s = fmaxf(s, old[y]);
                if (s != old[y])
                    rescale_rows(A.pages[y] + ((int64_t)p * A.hkv + h) * A.page * D, row0 * (D / 16), old[y] / s, lane, 32);
            }
            if (lane == 0) A.scale[y][(int64_t)p * A.hkv + h] = s;
            inv[y] = 1.f / s;
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) f[y][i] = fabsf(f[y][i]) < INFINITY ? f[y][i] * inv[y] : NAN;
        }
        uint8_t* o = A.pages[0] + base;
        uint8_t* ov = A.pages[1] + base + 2 * s0;
        if constexpr (N == 2) {
            *reinterpret_cast<uint16_t*>(o + ca) = f32x2_to_e4m3x2(f[0][0], f[0][1]);
            *reinterpret_cast<uint16_t*>(o + cb) = f32x2_to_e4m3x2(f[0][2], f[0][3]);
            *reinterpret_cast<uint32_t*>(ov) = (uint32_t)f32x2_to_e4m3x2(f[1][0], f[1][1]) | (uint32_t)f32x2_to_e4m3x2(f[1][2], f[1][3]) << 16;
        } else {
            const uint16_t two = f32x2_to_e4m3x2(f[0][0], f[0][1]);
            o[ca] = (uint8_t)two;
            o[cb] = (uint8_t)(two >> 8);
            *reinterpret_cast<uint16_t*>(ov) = f32x2_to_e4m3x2(f[1][0], f[1][1]);
        }
    }
}

template <int D, bool FP8, int MAXU, int MAXT, bool AHEAD>
cudaError_t append_pages_launch(const AppendArgs& A, int64_t ctas, int threads, cudaStream_t s) {
    constexpr int smem = AHEAD ? 4 * MAXU * MAXT * (int)sizeof(float4) : 0;
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> done{0};
        if (first_on_device(done)) {
            const cudaError_t e = cudaFuncSetAttribute(append_pages_kernel<D, FP8, MAXU, MAXT, AHEAD>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            mark_on_device(done);
        }
    }
    return launch_dependent(append_pages_kernel<D, FP8, MAXU, MAXT, AHEAD>, dim3((unsigned)ctas), threads, smem, s, 0, A);
}

// 16-value units of a page over 64 to 512 threads, 1 or 2 to a thread.  Rows of e4m3 pages are fetched a head ahead
// where a CTA has several heads (16391 tokens x 8 heads, q in a kernel of its own then, pages of 16 / 32 / 64: 75.5 -> 69.3,
// 77.8 -> 70.8, 69.5 -> 65.5 us; with one head 2000 tokens took 13.4 for 12.4); bf16 pages, which wait for no scale, gain
// nothing by it (70.3 -> 71.4, 70.3 -> 72.9, 70.4 -> 69.0).  Pages of 128 rows in 256 threads of 4 units would take 206
// registers.
int append_threads(int page, int d) {
    const int units = page * (d / 16);
    return units > 512 ? 512 : std::min(APP_THREADS, units);
}
template <int D, bool FP8>
cudaError_t append_pages(const AppendArgs& A, int64_t ctas, cudaStream_t s) {
    const int units = A.page * (D / 16), nt = append_threads(A.page, D);
    const bool ahead = FP8 && A.run > 1;
    if constexpr (D == 128)
        if (nt == 512)
            return ahead ? append_pages_launch<D, FP8, 2, 512, FP8>(A, ctas, nt, s) : append_pages_launch<D, FP8, 2, 512, false>(A, ctas, nt, s);
    if (units > nt)
        return ahead ? append_pages_launch<D, FP8, 2, APP_THREADS, FP8>(A, ctas, nt, s) : append_pages_launch<D, FP8, 2, APP_THREADS, false>(A, ctas, nt, s);
    return ahead ? append_pages_launch<D, FP8, 1, APP_THREADS, FP8>(A, ctas, nt, s) : append_pages_launch<D, FP8, 1, APP_THREADS, false>(A, ctas, nt, s);
}

int rope_heads_per_thread(int64_t n, int heads);

}  // namespace kvo

extern "C" kvo_status kvo_paged_append(const kvo_paged_cache* cache, const void* k, int64_t k_token_stride,
                                       const void* v, int64_t v_token_stride, int64_t tokens, const int32_t* cu,
                                       const int32_t* start, const uint64_t* freq, int rot_dim, int interleaved,
                                       float amplitude, const void* q, int64_t q_token_stride, int n_q_heads,
                                       void* q_out, void* k_out, int32_t* status, kvo_stream_t stream) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (const char* m = paged_cache_error(cache)) return bad(m);
    if (tokens < 0 || tokens > INT32_MAX) return bad("tokens must be in 0..2^31 - 1");
    if (tokens == 0 || (cache->batch == 0 && cu)) return KVO_OK;
    if (!cu && tokens != cache->batch) return bad("without cu every request appends one token: tokens must equal batch");
    if (!k || !v || !start) return bad("null k, v or start");
    const int D = cache->head_dim, hkv = cache->n_kv_heads;
    if (freq && (rot_dim < 16 || rot_dim % 16 || rot_dim > D)) return bad("rot_dim must be a multiple of 16 in 16..head_dim");
    if (q && (!q_out || n_q_heads < 1 || n_q_heads > 4096)) return bad("q needs q_out and n_q_heads in 1..4096");
    for (const void* p : {k, v, q, (const void*)q_out, (const void*)k_out})
        if ((uintptr_t)p % 16) return bad("k, v, q, q_out and k_out must be 16-byte aligned");
    if (k_token_stride % 8 || v_token_stride % 8 || q_token_stride % 8) return bad("strides must be multiples of 8 elements");
    // an output is its input in place, row for row, or apart from everything that the call reads
    struct Rows { const void* at; int64_t stride, len; } in[3] = {{k, k_token_stride, (int64_t)hkv * D},
                                                                  {v, v_token_stride, (int64_t)hkv * D},
                                                                  {q, q_token_stride, (int64_t)n_q_heads * D}};
    struct Out { void* at; int64_t len; int own; } out[2] = {{k_out, (int64_t)hkv * D, 0}, {q ? q_out : nullptr, (int64_t)n_q_heads * D, 2}};
    for (const Out& o : out)
        for (int i = 0; o.at && i < 3; ++i) {
            if (!in[i].at || !ranges_meet(o.at, 2 * tokens * o.len, in[i].at, rows_bytes(tokens, in[i].stride, in[i].len))) continue;
            if (i != o.own || o.at != in[i].at || (tokens > 1 && in[i].stride != o.len))
                return bad("k_out and q_out must be apart from the inputs, or k and q themselves where those are contiguous");
        }
    if (k_out && q && ranges_meet(k_out, 2 * tokens * out[0].len, q_out, 2 * tokens * out[1].len))
        return bad("k_out and q_out must not overlap");
    const int64_t pool = page_bytes(cache), scales = scale_bytes(cache), b = cache->batch;
    if (ranges_meet(cache->k_pages, pool, cache->v_pages, pool) || ranges_meet(cache->k_scale, scales, cache->v_scale, scales))
        return bad("K and V need pages and scales of their own");
    for (const Out& o : out)
        if (meets_any({o.at, 2 * tokens * o.len},
                      {{cache->k_pages, pool}, {cache->v_pages, pool}, {cache->k_scale, scales}, {cache->v_scale, scales},
                       {cache->table, 4 * b * cache->max_pages}, {start, 4 * b}, {cu, 4 * (b + 1)}, {freq, 4ll * rot_dim}}))
            return bad("k_out and q_out must share memory with nothing else that the call reads or writes");

    AppendArgs A{};
    A.pages[0] = (uint8_t*)cache->k_pages;
    A.pages[1] = (uint8_t*)cache->v_pages;
    A.scale[0] = cache->k_scale;
    A.scale[1] = cache->v_scale;
    A.table = cache->table;
    A.x[0] = (const uint16_t*)k;
    A.x[1] = (const uint16_t*)v;
    A.x_tok[0] = k_token_stride;
    A.x_tok[1] = v_token_stride;
    A.cu = cu;
    A.start = start;
    A.q = (const uint16_t*)q;
    A.q_out = (uint16_t*)q_out;
    A.k_out = (uint16_t*)k_out;
    A.status = status;
    A.tokens = tokens;
    A.q_tok = q_token_stride;
    A.batch = cache->batch;
    A.hkv = hkv;
    A.hq = n_q_heads;
    A.page = cache->page_size;
    A.n_pages = cache->n_pages;
    A.max_pages = cache->max_pages;
    A.R = RopeArgs{(const unsigned long long*)freq, freq ? rot_dim : 0, interleaved ? 1 : 0, amplitude};
    const bool fp8 = cache->format == KVO_PAGES_E4M3;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (!cu) {
        const int64_t warps = (int64_t)cache->batch * (hkv + (q ? n_q_heads : 0)), blocks = (warps + STEP_WARPS - 1) / STEP_WARPS;
        if (blocks > INT32_MAX) return bad("too many tokens");
        const dim3 grid((unsigned)blocks);
        const int nt = STEP_WARPS * 32;
        if (D == 128) e = fp8 ? launch_dependent(append_step_kernel<128, true>, grid, nt, 0, s, 0, A) : launch_dependent(append_step_kernel<128, false>, grid, nt, 0, s, 0, A);
        else e = fp8 ? launch_dependent(append_step_kernel<64, true>, grid, nt, 0, s, 0, A) : launch_dependent(append_step_kernel<64, false>, grid, nt, 0, s, 0, A);
    } else {
        const int64_t units = tokens / cache->page_size + 2 * (int64_t)cache->batch;
        if (units * hkv > INT32_MAX / 2) return bad("too many tokens");
        // The offsets and the angles of a page's rows cost about as much as one head's rest: where there are pages
        // enough to fill the device, a CTA takes up to 8 heads with them (16391 tokens x 8 heads, e4m3, with q: 80.5 us
        // at 1 head, 73.2 at 2, 70.4 at 4, 68.5 at 8, before rows were fetched ahead), and likewise where many requests touch
        // many pages (100 requests of 7 tokens 17.9 us at 1 head, 13.4 at 3, 16.6 at 7).
        A.run = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(hkv, 8), std::max(tokens / cache->page_size * hkv / 228, units * hkv / 456)));
        A.runs = (hkv + A.run - 1) / A.run;
        A.page_ctas = (int)(units * A.runs);
        int64_t ctas = A.page_ctas;
        if (q) {
            const int64_t n = tokens * (D / 16), threads = append_threads(A.page, D);
            A.q_per = rope_heads_per_thread(n, n_q_heads);
            A.q_blocks = (int)((n + threads - 1) / threads);
            ctas += (int64_t)A.q_blocks * ((n_q_heads + A.q_per - 1) / A.q_per);
            if (ctas > INT32_MAX) return bad("too many tokens");
        }
        if (D == 128) e = fp8 ? append_pages<128, true>(A, ctas, s) : append_pages<128, false>(A, ctas, s);
        else e = fp8 ? append_pages<64, true>(A, ctas, s) : append_pages<64, false>(A, ctas, s);
    }
    if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    return KVO_OK;
}
