// The softmax passes over a 128-column row of scores in TMEM (thread = row) that
// the forward and the shared prefix's kernel have in common.
#pragma once

#include "fa_ptx.cuh"

namespace fa {

// Pass 1 over one 128-column S row in TMEM (thread = row): the maximum of the
// raw scores.  Chunks of 32 columns are double-buffered (the next loads while
// this one is scanned).  MASKED: columns c > lim2 or c < lo2 are excluded;
// instantiated only for the blocks that hold a masked column.
template <bool MASKED>
__device__ __forceinline__ float row_max_pass(uint32_t taddr, int lim2, int lo2) {
    // eight running maxima, so that the 64 max instructions form eight short dependency chains
    float mx[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
    uint32_t va[32], vb[32];
    tmem_ld32_async(taddr, va);
    tmem_wait_ld(va);
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
        uint32_t(&v)[32] = (q4 & 1) ? vb : va;
        uint32_t(&nx)[32] = (q4 & 1) ? va : vb;
        if (q4 + 1 < 4) tmem_ld32_async(taddr + (q4 + 1) * 32, nx);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float x0 = __uint_as_float(v[i]), x1 = __uint_as_float(v[i + 1]);
            if constexpr (MASKED) {
                if (q4 * 32 + i > lim2 || q4 * 32 + i < lo2) x0 = -INFINITY;
                if (q4 * 32 + i + 1 > lim2 || q4 * 32 + i + 1 < lo2) x1 = -INFINITY;
            }
            mx[(i >> 1) & 7] = fmax3(mx[(i >> 1) & 7], x0, x1);
        }
        if (q4 + 1 < 4) tmem_wait_ld(nx);
    }
    return fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], fmax3(mx[5], mx[6], mx[7])));
}

// Pass 2: p = 2^(s c - m) for the 128 columns, their sum, and bf16 P written
// to paddr: either over the S columns already read (paddr = taddr: keys
// [32 q, 32 q + 32) to columns [16 q, 16 q + 16); the load in flight is always
// of columns >= 32 (q + 1)), or to columns of its own.
template <bool MASKED>
__device__ __forceinline__ float exp_pass(uint32_t taddr, uint32_t paddr, int lim2, int lo2, float c, float msub) {
    float2 rs[4];  // four partial sums (short dependency chains), added at the end
#pragma unroll
    for (int k = 0; k < 4; ++k) rs[k] = make_float2(0.f, 0.f);
    const float2 c2 = make_float2(c, c), nm2 = make_float2(-msub, -msub);
    uint32_t va[32], vb[32];
    tmem_ld32_async(taddr, va);
    tmem_wait_ld(va);
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
        uint32_t(&v)[32] = (q4 & 1) ? vb : va;
        uint32_t(&nx)[32] = (q4 & 1) ? va : vb;
        if (q4 + 1 < 4) tmem_ld32_async(taddr + (q4 + 1) * 32, nx);
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = __uint_as_float(v[2 * i]), s1 = __uint_as_float(v[2 * i + 1]);
            if constexpr (MASKED) {
                if (q4 * 32 + 2 * i > lim2 || q4 * 32 + 2 * i < lo2) s0 = -INFINITY;
                if (q4 * 32 + 2 * i + 1 > lim2 || q4 * 32 + 2 * i + 1 < lo2) s1 = -INFINITY;
            }
            const float2 x = ffma2(make_float2(s0, s1), c2, nm2);  // s*c - m, two lanes
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            rs[i & 3] = fadd2(rs[i & 3], e);
            pk[i] = pack_bf16(e.x, e.y);
        }
        tmem_st16_async(paddr + q4 * 16, pk);
        if (q4 + 1 < 4) tmem_wait_ld(nx);
    }
    tmem_wait_st();
    const float2 r01 = fadd2(rs[0], rs[1]), r23 = fadd2(rs[2], rs[3]);
    return (r01.x + r23.x) + (r01.y + r23.y);
}

}  // namespace fa
