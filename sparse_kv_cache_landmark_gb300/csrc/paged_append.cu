// kvo_paged_append: new keys and values into a paged cache, keys (and the
// queries beside them) rotated on the way.
//
// A key is rotated in fp32 and rounded once to bf16: that value goes to k_out
// and to bf16 pages, and it is what e4m3 pages quantise.  The one rounding
// step before the quantisation (2^-9 relative against e4m3's 2^-4) makes the
// prompt's own attention and the cache agree on what the key is.
//
// One CTA owns one (page, KV head) that the call touches, so the page's scale
// needs no atomics: it holds the page's new rows in registers, takes their
// largest magnitude, settles the scale, moves rows of earlier calls to it when
// it grew, and writes codes.  Further CTAs of the same launch rotate q.
//
// Bound by HBM on prompts (k and v read once, pages and k_out written once)
// and by one chain of dependent loads on a decode step.
#include <stdio.h>

#include <algorithm>

#include "launch.cuh"
#include "paged.cuh"
#include "rope.cuh"

namespace kvo {

constexpr int APP_THREADS = 256;

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
    int units;                    // upper bound of the pages touched
    int q_per;                    // query heads per thread
    RopeArgs R;
};

__device__ __forceinline__ void set_status(int32_t* status, int bits) {
    if (status && bits) atomicOr(status, bits);
}

// Request b's token range; false (with a status bit) when the caller's offsets
// leave [0, tokens] or the start is negative.
__device__ __forceinline__ bool request_range(const AppendArgs& A, int b, int64_t& t0, int64_t& n, int& start) {
    t0 = A.cu ? A.cu[b] : b;
    n = A.cu ? (int64_t)A.cu[b + 1] - t0 : 1;
    start = A.start[b];
    return t0 >= 0 && n >= 0 && t0 + n <= A.tokens && start >= 0;
}

template <int D, bool FP8, int MAXU>
__device__ __forceinline__ void append_page(const AppendArgs& A) {
    constexpr int UNITS = D / 16;                       // 16-value units of a row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int u = blockIdx.x / A.hkv, h = blockIdx.x - u * A.hkv;
    __shared__ float red[2][APP_THREADS / 32];

    if (blockIdx.x == 0 && A.status)                    // bad offsets of any request, also of one that no unit reaches
        for (int i = tid; i < A.batch; i += APP_THREADS) {
            int64_t t0, n;
            int start;
            if (!request_range(A, i, t0, n, start)) set_status(A.status, KVO_DEV_BAD_COUNT);
        }
    // Request b has at most floor(n / page) + 2 touched pages, so its units start
    // at floor(cu[b] / page) + 2 b: every request finds its own without a scan.
    int b = u, j = 0;
    if (A.cu) {
        auto first = [&](int i) { return (int64_t)max(__ldg(A.cu + i), 0) / A.page + 2 * (int64_t)i; };
        b = warp_find(A.batch, u, first);
        j = u - (int)first(b);
    }
    int64_t t0, n;
    int start;
    if (!request_range(A, b, t0, n, start)) return;
    const int64_t at = start / A.page + (int64_t)j;       // logical page
    const int64_t pos0 = max((int64_t)start, at * A.page), pos1 = min(start + n, (at + 1) * A.page);
    if (pos0 >= pos1) return;
    if (at >= A.max_pages) {
        if (tid == 0 && h == 0) set_status(A.status, KVO_DEV_BAD_COUNT);
        return;
    }
    const int p = A.table[(int64_t)b * A.max_pages + at];
    if (p < 0 || p >= A.n_pages) {
        if (tid == 0 && h == 0) set_status(A.status, KVO_DEV_BAD_BLOCK_ID);
        return;
    }
    const int row0 = (int)(pos0 - at * A.page), rows = (int)(pos1 - pos0);
    const int64_t tok0 = t0 + (pos0 - start);

    uint4 xa[2][MAXU], xb[2][MAXU];
#pragma unroll
    for (int i = 0; i < MAXU; ++i) {
        const int w = tid + i * APP_THREADS, r = w / UNITS, un = w % UNITS;
        if (r < rows) {
            int ca, cb;
            rope_chunks(A.R, D, un, ca, cb);
            const uint16_t* k = A.x[0] + (tok0 + r) * A.x_tok[0] + (int64_t)h * D;
            const uint16_t* v = A.x[1] + (tok0 + r) * A.x_tok[1] + (int64_t)h * D;
            xa[0][i] = *reinterpret_cast<const uint4*>(k + ca);
            xb[0][i] = *reinterpret_cast<const uint4*>(k + cb);
            xa[1][i] = *reinterpret_cast<const uint4*>(v + ca);
            xb[1][i] = *reinterpret_cast<const uint4*>(v + cb);
        }
    }
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < MAXU; ++i) {
        const int w = tid + i * APP_THREADS, r = w / UNITS, un = w % UNITS;
        if (r >= rows) continue;
        float c[8], s[8];
        if (rope_unit(A.R, un, (int)(pos0 + r), c, s)) rope_rotate(A.R.interleaved, c, s, xa[0][i], xb[0][i]);
        if (A.k_out) {
            int ca, cb;
            rope_chunks(A.R, D, un, ca, cb);
            uint16_t* o = A.k_out + ((tok0 + r) * A.hkv + h) * D;
            *reinterpret_cast<uint4*>(o + ca) = xa[0][i];
            *reinterpret_cast<uint4*>(o + cb) = xb[0][i];
        }
        if (FP8) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint4& src = e < 4 ? xa[x][i] : xb[x][i];
                    const uint32_t word = reinterpret_cast<const uint32_t*>(&src)[e & 3];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float f = fabsf(half ? __uint_as_float(word & 0xFFFF0000u) : __uint_as_float(word << 16));
                        if (f < INFINITY) top[x] = fmaxf(top[x], f);
                    }
                }
        }
    }
    float inv[2];
    if (FP8) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int o = 16; o; o >>= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], o));
            if (lane == 0) red[x][warp] = top[x];
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < APP_THREADS / 32; ++i) m = fmaxf(m, red[x][i]);
            float s = e4m3_scale(m);
            float* slot = A.scale[x] + (int64_t)p * A.hkv + h;
            if (row0 > 0) {                                // rows of earlier calls: the scale never shrinks
                const float old = *slot;
                s = fmaxf(s, old);
                if (s != old) {
                    const float ratio = old / s;
                    uint4* row = reinterpret_cast<uint4*>(A.pages[x] + ((int64_t)p * A.hkv + h) * A.page * D);
                    for (int w = tid; w < row0 * UNITS; w += APP_THREADS) {
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
            }
            inv[x] = 1.f / s;
            top[x] = s;
        }
        __syncthreads();                                   // every thread has read the old scale
        if (tid == 0)
#pragma unroll
            for (int x = 0; x < 2; ++x) A.scale[x][(int64_t)p * A.hkv + h] = top[x];
    }
#pragma unroll
    for (int i = 0; i < MAXU; ++i) {
        const int w = tid + i * APP_THREADS, r = w / UNITS, un = w % UNITS;
        if (r >= rows) continue;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            int ca, cb;
            rope_chunks(A.R, D, un, ca, cb);
            const int64_t base = (((int64_t)p * A.hkv + h) * A.page + row0 + r) * D;
            if (!FP8) {
                uint16_t* o = reinterpret_cast<uint16_t*>(A.pages[x]) + base;
                *reinterpret_cast<uint4*>(o + ca) = xa[x][i];
                *reinterpret_cast<uint4*>(o + cb) = xb[x][i];
            } else {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t* word = reinterpret_cast<const uint32_t*>(half ? &xb[x][i] : &xa[x][i]);
                    uint32_t codes[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float lo = __uint_as_float(word[e] << 16), hi = __uint_as_float(word[e] & 0xFFFF0000u);
                        // an infinity has no code: NaN keeps it visible (saturation would turn it into 448 s)
                        lo = fabsf(lo) < INFINITY ? lo * inv[x] : NAN;
                        hi = fabsf(hi) < INFINITY ? hi * inv[x] : NAN;
                        const uint32_t two = f32x2_to_e4m3x2(lo, hi);
                        codes[e >> 1] = (e & 1) ? codes[e >> 1] | (two << 16) : two;
                    }
                    *reinterpret_cast<uint2*>(A.pages[x] + base + (half ? cb : ca)) = make_uint2(codes[0], codes[1]);
                }
            }
        }
    }
}

// Blocks [0, units * Hkv): pages.  The rest: q.
template <int D, bool FP8, int MAXU>
__global__ void __launch_bounds__(APP_THREADS) append_pages_kernel(const __grid_constant__ AppendArgs A) {
    grid_wait();
    const int kv_blocks = A.units * A.hkv;
    if ((int)blockIdx.x < kv_blocks) {
        append_page<D, FP8, MAXU>(A);
        return;
    }
    constexpr int UNITS = D / 16;
    const int64_t i = (int64_t)(blockIdx.x - kv_blocks) * APP_THREADS + threadIdx.x;
    const int64_t per_split = (A.tokens * UNITS + APP_THREADS - 1) / APP_THREADS * APP_THREADS;
    const int64_t split = i / per_split, k = i - split * per_split;
    if (k >= A.tokens * UNITS) return;
    const int64_t t = k / UNITS;
    const int u = (int)(k - t * UNITS);
    int b = (int)t;
    if (A.cu) {
        int lo = 0, hi = A.batch;                          // the last b with cu[b] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (__ldg(A.cu + mid) <= t) lo = mid; else hi = mid;
        }
        b = lo;
    }
    int64_t t0, n;
    int start;
    if (!request_range(A, b, t0, n, start) || t < t0 || t >= t0 + n) return;
    const int h0 = (int)split * A.q_per, h1 = min(A.hq, h0 + A.q_per);
    rope_heads(A.R, D, A.q + t * A.q_tok, D, A.q_out + t * A.hq * D, D, u, (int)(start + (t - t0)), h0, h1);
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
    if (tokens == 0 || cache->batch == 0) return KVO_OK;
    if (!k || !v || !start) return bad("null k, v or start");
    if (!cu && tokens != cache->batch) return bad("without cu every request appends one token: tokens must equal batch");
    const int D = cache->head_dim, hkv = cache->n_kv_heads;
    if (freq && (rot_dim < 16 || rot_dim % 16 || rot_dim > D)) return bad("rot_dim must be a multiple of 16 in 16..head_dim");
    if (q && (!q_out || n_q_heads < 1 || n_q_heads > 4096)) return bad("q needs q_out and n_q_heads in 1..4096");
    for (const void* p : {k, v, q, (const void*)q_out, (const void*)k_out})
        if ((uintptr_t)p % 16) return bad("k, v, q, q_out and k_out must be 16-byte aligned");
    if (k_token_stride % 8 || v_token_stride % 8 || q_token_stride % 8) return bad("strides must be multiples of 8 elements");

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
    const int64_t units = cu ? tokens / cache->page_size + 2 * (int64_t)cache->batch : cache->batch;
    A.units = (int)units;
    int64_t blocks = units * hkv;
    if (q) {
        const int64_t n = tokens * (D / 16);
        A.q_per = rope_heads_per_thread(n, n_q_heads);
        blocks += (n + APP_THREADS - 1) / APP_THREADS * ((n_q_heads + A.q_per - 1) / A.q_per);
    }
    if (blocks > INT32_MAX) return bad("too many tokens");
    const bool fp8 = cache->format == KVO_PAGES_E4M3;
    // rows x 16-value units of a page over 256 threads; without cu a page takes one row
    const int per_page = (cu ? cache->page_size : 1) * (D / 16);
    const int maxu = per_page <= APP_THREADS ? 1 : per_page <= 2 * APP_THREADS ? 2 : 4;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
#define KVO_APPEND(D_, F_, U_) e = launch_dependent(append_pages_kernel<D_, F_, U_>, dim3((unsigned)blocks), APP_THREADS, 0, s, 0, A)
#define KVO_APPEND_U(D_, F_)                                                                  \
    do {                                                                                      \
        if (maxu == 1) KVO_APPEND(D_, F_, 1); else if (maxu == 2) KVO_APPEND(D_, F_, 2);      \
        else KVO_APPEND(D_, F_, 4);                                                           \
    } while (0)
    if (D == 128) { if (fp8) KVO_APPEND_U(128, true); else KVO_APPEND_U(128, false); }
    else { if (fp8) KVO_APPEND_U(64, true); else KVO_APPEND_U(64, false); }
#undef KVO_APPEND_U
#undef KVO_APPEND
    if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    return KVO_OK;
}
