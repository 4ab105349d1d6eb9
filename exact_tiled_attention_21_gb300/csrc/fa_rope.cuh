// Rotary positions: what the rotation kernel and the cache append share.
//
// Pair i of a head turns by pos * f_i radians.  The frequencies come as turns
// per position, in units of 2^-64 turn: pos * turns mod 2^64 is then the exact
// fraction of a turn for every 32-bit position, in one 64-bit integer product
// (what is left is the table's own 2^-52 pos f_i), where pos * f_i in fp32 is off
// by up to 2^-24 pos f_i radians (0.008 at position 131072), and fp64 has no
// throughput to speak of on this GPU.
#pragma once

#include "fa_ptx.cuh"

namespace fa {

// cos and sin of a fraction of a turn, times mag: the nearest quarter turn
// comes off in integers, which leaves an angle of at most pi / 4 exactly (to
// 2^-32 turn), held in two floats; the Taylor polynomials to x^9 and x^10 are
// within 2^-29 there, and the large terms are added last, with what their
// rounding left, so that 19 of 20 results are the correctly rounded ones and
// all are within 2^-23.9.  The hardware's sine and cosine (2^-20.5), and sums
// of 2^-23, flip enough bf16 roundings to show in the cache's bytes.
__device__ __forceinline__ void turn_cos_sin(int pos, uint64_t turns, float mag, float& c, float& s) {
    const uint32_t t = (uint32_t)(((uint64_t)(int64_t)pos * turns) >> 32);
    const uint32_t q = (t + 0x20000000u) >> 30;
    const int r = (int)(t - (q << 30));                      // |r| <= 2^29
    constexpr float kHi = 1.4629180792671596e-09f;           // 2 pi / 2^32 as two floats
    constexpr float kLo = (float)(1.4629180792671596e-09 - (double)kHi);
    const float rh = (float)(r & ~0xFF), rl = (float)(r & 0xFF);  // both exact
    const float a = rh * kHi;
    const float lo = fmaf(rl, kHi, fmaf(rh, kLo, fmaf(rh, kHi, -a)));
    const float z = a * a, ze = fmaf(a, a, -z), hz = 0.5f * z;
    const float ps = fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
    const float pc = fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f);
    const float sn = a + fmaf(a * z, ps, fmaf(lo, -hz, lo));                   // sin a + lo cos a
    const float one = 1.f - hz, left = (1.f - one) - hz;
    const float cs = one + (left + fmaf(z * z, pc, fmaf(-0.5f, ze, -(lo * a))));  // cos a - lo sin a
    c = __uint_as_float(__float_as_uint((q & 1) ? sn : cs) ^ (((q + 1) & 2) << 30)) * mag;
    s = __uint_as_float(__float_as_uint((q & 1) ? cs : sn) ^ ((q & 2) << 30)) * mag;
}

// The same for the eight pairs of one task (turns: 16-byte aligned).
__device__ __forceinline__ void task_cos_sin(int pos, const uint64_t* turns, float mag, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 f = reinterpret_cast<const ulonglong2*>(turns)[i];
        turn_cos_sin(pos, f.x, mag, c[2 * i], s[2 * i]);
        turn_cos_sin(pos, f.y, mag, c[2 * i + 1], s[2 * i + 1]);
    }
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Rotates eight pairs held in two 16-byte pieces of a row, in fp32, rounded to
// bf16 once.  INTER: the pieces are 16 consecutive columns, pair i in columns
// 2i, 2i + 1.  Otherwise a holds the first members and b the second ones.
template <bool INTER>
__device__ __forceinline__ void rotate16(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
    uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
    uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x1 = bf_lo(wa[i]), x2 = bf_hi(wa[i]);
            wa[i] = pack_bf16(fmaf(x1, c[i], -(x2 * s[i])), fmaf(x2, c[i], x1 * s[i]));
            const float y1 = bf_lo(wb[i]), y2 = bf_hi(wb[i]);
            wb[i] = pack_bf16(fmaf(y1, c[4 + i], -(y2 * s[4 + i])), fmaf(y2, c[4 + i], y1 * s[4 + i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x1 = bf_lo(wa[i]), y1 = bf_hi(wa[i]), x2 = bf_lo(wb[i]), y2 = bf_hi(wb[i]);
            wa[i] = pack_bf16(fmaf(x1, c[2 * i], -(x2 * s[2 * i])), fmaf(y1, c[2 * i + 1], -(y2 * s[2 * i + 1])));
            wb[i] = pack_bf16(fmaf(x2, c[2 * i], x1 * s[2 * i]), fmaf(y2, c[2 * i + 1], y1 * s[2 * i + 1]));
        }
    }
}

// The columns of task p (of d / 16) of a row: two pieces of eight columns that
// hold eight pairs, or 16 columns behind the rotated part.
template <bool INTER>
__device__ __forceinline__ void task_columns(int p, int rot, int& c0, int& c1) {
    if (INTER || p >= rot / 16) {
        c0 = p * 16;
        c1 = c0 + 8;
    } else {
        c0 = p * 8;
        c1 = rot / 2 + c0;
    }
}

}  // namespace fa
