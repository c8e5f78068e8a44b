// kvo_rope: rotary positions of packed heads (the mathematics is in rope.cuh).
//
// Bound by HBM: every value is read and written once (4 bytes per value), and
// the angle of a (token, pair) is shared by all heads.  A thread owns 16 values
// (8 pairs) of one token, computes their 8 cosines and sines once and walks the
// token's heads with four heads' loads in flight.  16411 tokens x 40 heads of 128:
// 52.3 us, 6.4 TB/s (0.94 of a measured copy); 16 tokens: 2.1 us.
#include <stdio.h>

#include <algorithm>

#include "kvo_internal.cuh"
#include "launch.cuh"
#include "rope.cuh"

namespace kvo {

constexpr int ROPE_THREADS = 256;

// grid.x: (token, unit) pairs; grid.y: runs of `heads_per` heads.
__global__ void __launch_bounds__(ROPE_THREADS)
rope_kernel(const uint16_t* x, int64_t x_tok, int64_t x_head, uint16_t* out, int64_t out_tok,
            int64_t out_head, const int32_t* __restrict__ pos, RopeArgs R, int d, int64_t n, int heads,
            int heads_per) {
    const int units = d / 16;
    const int64_t i = (int64_t)blockIdx.x * ROPE_THREADS + threadIdx.x;
    if (i >= n) return;
    const int64_t t = i / units;
    const int u = (int)(i - t * units);
    const int h0 = blockIdx.y * heads_per, h1 = min(heads, h0 + heads_per);
    grid_wait();
    rope_heads(R, d, x + t * x_tok, x_head, out + t * out_tok, out_head, u, __ldg(pos + t), h0, h1);
}

// Heads a thread takes: 8 sincos (about 300 instructions) are spread over them, so as many as leave each SM 128 threads,
// up to 8 (two batches of loads).  With 2048 threads an SM instead 500 tokens of 40 heads took 6.5 us for 4.7, 2000 10.8
// for 8.0; with 32, 128 tokens 4.5 for 3.2.
int rope_heads_per_thread(int64_t n, int heads) {
    const int64_t want = 152 * 128;
    const int64_t splits = (want + n - 1) / n;
    return (int)std::max<int64_t>(1, std::min<int64_t>(8, heads / std::max<int64_t>(1, splits)));
}

// Which memory rows share.  A view has rows of d values at t * tok + h * head, t < T, h < H; strides of any size.
typedef __int128 wide;
struct RopeView {
    const void* at;
    int64_t tok, head;
};
// Whether m * step lies between lo and hi, both excluded, for some |m| < n.
bool multiple_between(wide lo, wide hi, int64_t step, int64_t n) {
    const wide s = step < 0 ? -(wide)step : (wide)step;
    if (s == 0 || n == 1) return lo < 0 && 0 < hi;
    const wide below = lo >= 0 ? lo / s : -((-lo + s - 1) / s);          // floor
    const wide m = std::max<wide>(below + 1, 1 - (wide)n);
    return m < n && m * s < hi;
}
// Whether two rows of the view share a value.
bool rope_rows_share(const RopeView& v, int64_t T, int H, int d) {
    if ((H == 1 || v.head >= d) && (T == 1 || v.tok >= (wide)(H - 1) * v.head + d)) return false;    // token after token
    if ((T == 1 || v.tok >= d) && (H == 1 || v.head >= (wide)(T - 1) * v.tok + d)) return false;     // head after head
    if (T > 1 && v.tok > -d && v.tok < d) return true;
    for (int h = 1; h < H; ++h)
        if (multiple_between(-d - (wide)h * v.head, d - (wide)h * v.head, v.tok, T)) return true;
    return false;
}
// Whether a row of x shares a value with a row of out.  Exact for equal strides; with equal token strides a token's heads
// are taken as one run, and with others all rows.
bool rope_views_meet(const RopeView& x, const RopeView& out, int64_t T, int H, int d) {
    const wide apart = ((wide)(intptr_t)out.at - (wide)(intptr_t)x.at) / 2;      // both are 16-byte aligned
    auto low = [](wide n, int64_t stride) { return stride < 0 ? n * stride : (wide)0; };
    auto high = [](wide n, int64_t stride) { return stride > 0 ? n * stride : (wide)0; };
    const wide x0 = low(H - 1, x.head), x1 = high(H - 1, x.head) + d;            // a token's heads
    const wide o0 = apart + low(H - 1, out.head), o1 = apart + high(H - 1, out.head) + d;
    if (o0 + low(T - 1, out.tok) >= x1 + high(T - 1, x.tok) || x0 + low(T - 1, x.tok) >= o1 + high(T - 1, out.tok)) return false;
    if (T > 1 && x.tok != out.tok) return true;
    if (H > 1 && x.head != out.head) return multiple_between(x0 - o1, x1 - o0, x.tok, T);
    for (int h = 1 - H; h < H; ++h)
        if (multiple_between(-d - apart - (wide)h * x.head, d - apart - (wide)h * x.head, x.tok, T)) return true;
    return false;
}

}  // namespace kvo

extern "C" kvo_status kvo_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
                               int64_t out_token_stride, int64_t out_head_stride, const int32_t* pos,
                               const uint64_t* freq, int64_t tokens, int heads, int head_dim, int rot_dim,
                               int interleaved, float amplitude, kvo_stream_t stream) {
    using namespace kvo;
    auto bad = [](const char* m) { set_last_error(m); return KVO_ERR_INVALID; };
    if (tokens < 0 || heads < 1) return bad("need tokens >= 0 and heads >= 1");
    if (heads > 65535) return bad("heads must be <= 65535");
    if (head_dim < 16 || head_dim % 16 || head_dim > 4096) return bad("head_dim must be a multiple of 16 in 16..4096");
    if (rot_dim < 16 || rot_dim % 16 || rot_dim > head_dim)
        return bad("rot_dim must be a multiple of 16 in 16..head_dim");
    if (tokens == 0) return KVO_OK;
    if (!x || !out || !pos || !freq) return bad("null pointer argument");
    if ((uintptr_t)x % 16 || (uintptr_t)out % 16) return bad("x and out must be 16-byte aligned");
    if (x_token_stride % 8 || x_head_stride % 8 || out_token_stride % 8 || out_head_stride % 8)
        return bad("strides must be multiples of 8 elements");
    if ((tokens > 1 && out_token_stride == 0) || (heads > 1 && out_head_stride == 0))
        return bad("rows of out must not share memory");
    if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
        return bad("in place needs equal strides");
    const RopeView in{x, x_token_stride, x_head_stride}, to{out, out_token_stride, out_head_stride};
    if (rope_rows_share(to, tokens, heads, head_dim)) return bad("rows of out must not share memory");
    if (x != out && rope_views_meet(in, to, tokens, heads, head_dim))
        return bad("out must be apart from x, or x itself with equal strides");
    const int units = head_dim / 16;
    if (tokens > (int64_t)INT32_MAX * ROPE_THREADS / units) return bad("too many tokens");
    const int64_t n = tokens * units;
    const int per = rope_heads_per_thread(n, heads);
    const RopeArgs R{(const unsigned long long*)freq, rot_dim, interleaved ? 1 : 0, amplitude};
    const dim3 grid((unsigned)((n + ROPE_THREADS - 1) / ROPE_THREADS), (unsigned)((heads + per - 1) / per));
    const cudaError_t e = launch_dependent(rope_kernel, grid, ROPE_THREADS, 0, (cudaStream_t)stream, 0, (const uint16_t*)x,
                                           x_token_stride, x_head_stride, (uint16_t*)out, out_token_stride,
                                           out_head_stride, pos, R, head_dim, n, heads, per);
    if (e != cudaSuccess) { set_last_error(cudaGetErrorString(e)); return KVO_ERR_CUDA; }
    return KVO_OK;
}
