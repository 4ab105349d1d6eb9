// e4m3 conversions and the mma / cp.async wrappers of the 8-bit cache kernels.
#pragma once

#include <cuda_fp16.h>

#include "fa_ptx.cuh"

namespace fa {

// Two e4m3 bytes (low half of w) as two halves: exact (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_half2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
}
// Four values to e4m3 bytes: nearest, ties to even, saturated at +-448, NaN kept.
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Whether a positive float is a power of two in the normal range.
__device__ __forceinline__ bool is_pow2(float s) {
    const uint32_t u = __float_as_uint(s);
    return (u & 0x807FFFFFu) == 0 && u - 0x00800000u < 0x7F000000u;
}

// Sixteen e4m3 bytes with scale `from` as e4m3 bytes with scale `to`, each
// value rounded to nearest once more.  Between powers of two, downwards, that
// is a product in fp16: it is exact wherever the result does not round to zero
// (four significant bits above 2^-14), 3 instructions for 2 values.  (40 with a
// division for each bound the eviction at 62 us of B = 32, 1024 of 4096 tokens.)
__device__ __forceinline__ uint4 e4m3_rescale16(uint4 x, float from, float to) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
    if (from <= to && is_pow2(from) && is_pow2(to)) {
        const int e = (int)(__float_as_uint(to) >> 23) - (int)(__float_as_uint(from) >> 23);
        const __half2 f = __float2half2_rn(__uint_as_float((uint32_t)(127 - min(e, 126)) << 23));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint16_t r[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t h = j ? e4m3x2_hi_to_half2(w[i]) : e4m3x2_to_half2(w[i]);
                const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h), f);
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r[j]) : "r"(*reinterpret_cast<const uint32_t*>(&p)));
            }
            w[i] = (uint32_t)r[0] | ((uint32_t)r[1] << 16);
        }
        return x;
    }
    const float by = __fdiv_rn(from, to);  // first: a value times a scale may overflow, or lose bits among the subnormals
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = half2_to_float2(e4m3x2_to_half2(w[i])), b = half2_to_float2(e4m3x2_hi_to_half2(w[i]));
        w[i] = e4m3x4(a.x * by, a.y * by, b.x * by, b.y * by);
    }
    return x;
}

// D (16 x 8, fp32) += A (16 x 16, f16) * B (16 x 8, f16), one warp.  With g = lane / 4, t = lane % 4:
// a = rows g, g + 8, g, g + 8 at columns 2t (+1) and 2t + 8 (+1); b = rows 2t (+1) and 2t + 8 (+1) of
// column g; d = rows g, g, g + 8, g + 8 at columns 2t, 2t + 1, 2t, 2t + 1.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements whose row g lane (g, t) holds columns 2t, 2t + 1 of.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Asynchronous copies to shared memory; `ok` = false fills with zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace fa
