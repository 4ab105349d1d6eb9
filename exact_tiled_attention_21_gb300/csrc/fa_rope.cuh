// Rotary positions: what the rotation kernel and the cache append share.
//
// Pair i of a head turns by pos * f_i radians.  The frequencies come as turns
// per position, in units of 2^-64 turn: pos * turns mod 2^64 is then the exact
// fraction of a turn for every 32-bit position, in one 64-bit integer product,
// where pos * f_i in fp32 is off by up to 2^-24 pos f_i radians (0.008 at
// position 131072), and fp64 has no throughput to speak of on this GPU.
#pragma once

#include "fa_ptx.cuh"

namespace fa {

// cos and sin of a fraction of a turn, times mag.  The top 32 bits, as a signed
// fraction in [-1/2, 1/2), lose at most 2^-25 turn in the fp32 conversion; the
// hardware sine and cosine are within 2^-20.5 on [-pi, pi].  Both are far below
// the half step of the bf16 result (2^-9), and cost 1/5 of the library pair.
__device__ __forceinline__ void turn_cos_sin(int pos, uint64_t turns, float mag, float& c, float& s) {
    const uint64_t t = (uint64_t)(int64_t)pos * turns;
    const float a = (float)(int32_t)(uint32_t)(t >> 32) * 1.4629180792671596e-09f;  // 2 pi / 2^32
    float cc, ss;
    asm("cos.approx.ftz.f32 %0, %1;" : "=f"(cc) : "f"(a));
    asm("sin.approx.ftz.f32 %0, %1;" : "=f"(ss) : "f"(a));
    c = cc * mag;
    s = ss * mag;
}

// The same for the eight pairs of one task (turns: 16-byte aligned).
__device__ __forceinline__ void task_cos_sin(int pos, const uint64_t* turns, float mag, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 f = __ldg(reinterpret_cast<const ulonglong2*>(turns) + i);
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
