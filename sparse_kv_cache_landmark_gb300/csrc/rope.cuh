// Rotary positions, shared by the rotation kernel and the paged append.
//
// A pair (u, v) of a head at position p turns by the angle 2 pi p f, f the
// pair's frequency in turns per position:
//     u' = amp (u cos - v sin),  v' = amp (u sin + v cos).
// f is held as an unsigned 64-bit fraction of a turn (units of 2^-64), so the
// integer product p * f modulo 2^64 IS the phase: whole turns wrap away
// exactly at every position, negative ones included, where p * f in 32-bit
// floats would be off by p * 2^-24 turns (6% of a turn at a million).  The top
// 32 bits become the argument of sincospif.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace kvo {

// A head is cut into units of 16 values, two chunks of 8 (16 bytes) half a part
// apart: unit u < rot_dim / 16 takes chunks 8 u and rot_dim / 2 + 8 u of the rotated
// part, the units after it the same of the rest.  Neighbouring lanes then touch
// neighbouring chunks in both pair layouts.
struct RopeArgs {
    const unsigned long long* freq;   // [rot_dim / 2]; NULL: nothing rotates
    int rot_dim;                      // a multiple of 16, <= head_dim (0 without freq)
    int interleaved;                  // 0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1)
    float amp;                        // factor on the rotated values
};

__device__ __forceinline__ void rope_sincos(int pos, unsigned long long f, float amp, float& c, float& s) {
    const unsigned long long ph = (unsigned long long)(long long)pos * f;
    // The nearest quarter turn is taken off as an integer, so the rest, at most an eighth of a turn, loses no more
    // than 2^-27 half turns as a float; then the angle is turned back by q quarters.
    const uint32_t top = (uint32_t)(ph >> 32);
    const uint32_t q = (top + 0x20000000u) >> 30;
    const float half_turns = (float)(int)(top - (q << 30)) * 4.656612873077393e-10f;    // 2^-31
    float s0, c0;
    sincospif(half_turns, &s0, &c0);
    const float sq = (q & 1) ? c0 : s0, cq = (q & 1) ? s0 : c0;
    s = (q & 2) ? -sq : sq;
    c = ((q + 1) & 2) ? -cq : cq;
    c *= amp;
    s *= amp;
}

// First value of the two chunks of unit u of a head of d values.
__device__ __forceinline__ void rope_chunks(const RopeArgs& R, int d, int u, int& a, int& b) {
    const int n = R.rot_dim / 16;
    if (u < n) {
        a = 8 * u;
        b = a + R.rot_dim / 2;
    } else {
        a = R.rot_dim + 8 * (u - n);
        b = a + (d - R.rot_dim) / 2;
    }
}

// cos and sin of the 8 pairs of unit u; returns false for a unit that passes through.
__device__ __forceinline__ bool rope_unit(const RopeArgs& R, int u, int pos, float (&c)[8], float (&s)[8]) {
    if (16 * u >= R.rot_dim) return false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // pairs 8u.. of the halves; interleaved: pairs 4u.. in chunk a, 4u.. of the second half of them in chunk b
        const int pair = !R.interleaved ? 8 * u + i : i < 4 ? 4 * u + i : R.rot_dim / 4 + 4 * u + i - 4;
        rope_sincos(pos, __ldg(R.freq + pair), R.amp, c[i], s[i]);
    }
    return true;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Rotates the two chunks of a unit in fp32, each result rounded once to bf16.
__device__ __forceinline__ void rope_rotate(bool interleaved, const float (&c)[8], const float (&s)[8], uint4& a,
                                            uint4& b) {
    uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
    uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float a0 = __uint_as_float(wa[w] << 16), a1 = __uint_as_float(wa[w] & 0xFFFF0000u);
        const float b0 = __uint_as_float(wb[w] << 16), b1 = __uint_as_float(wb[w] & 0xFFFF0000u);
        if (interleaved) {        // (a0, a1) is pair w, (b0, b1) pair 4 + w
            wa[w] = pack_bf16(a0 * c[w] - a1 * s[w], a0 * s[w] + a1 * c[w]);
            wb[w] = pack_bf16(b0 * c[4 + w] - b1 * s[4 + w], b0 * s[4 + w] + b1 * c[4 + w]);
        } else {                  // (a0, b0) is pair 2w, (a1, b1) pair 2w + 1
            wa[w] = pack_bf16(a0 * c[2 * w] - b0 * s[2 * w], a1 * c[2 * w + 1] - b1 * s[2 * w + 1]);
            wb[w] = pack_bf16(a0 * s[2 * w] + b0 * c[2 * w], a1 * s[2 * w + 1] + b1 * c[2 * w + 1]);
        }
    }
}

// One thread's part of rotating packed heads: unit u of one token, heads h0, h0 + 1, .. h1 - 1.
// x and out point at the token.  In place (out == x with equal strides) is allowed: each
// unit is read whole before it is written, by the thread that owns it.
__device__ __forceinline__ void rope_heads(const RopeArgs& R, int d, const uint16_t* x, int64_t x_head,
                                           uint16_t* out, int64_t out_head, int u, int pos, int h0, int h1) {
    float c[8], s[8];
    const bool rot = rope_unit(R, u, pos, c, s);
    int ca, cb;
    rope_chunks(R, d, u, ca, cb);
    constexpr int IN_FLIGHT = 4;
    for (int h = h0; h < h1; h += IN_FLIGHT) {
        uint4 a[IN_FLIGHT], b[IN_FLIGHT];
#pragma unroll
        for (int i = 0; i < IN_FLIGHT; ++i)
            if (h + i < h1) {
                a[i] = *reinterpret_cast<const uint4*>(x + (h + i) * x_head + ca);
                b[i] = *reinterpret_cast<const uint4*>(x + (h + i) * x_head + cb);
            }
#pragma unroll
        for (int i = 0; i < IN_FLIGHT; ++i)
            if (h + i < h1) {
                if (rot) rope_rotate(R.interleaved, c, s, a[i], b[i]);
                *reinterpret_cast<uint4*>(out + (h + i) * out_head + ca) = a[i];
                *reinterpret_cast<uint4*>(out + (h + i) * out_head + cb) = b[i];
            }
    }
}

}  // namespace kvo
