// Rotary positions on a [B, H, N, d] tensor of any strides (and their gradient,
// which is the rotation by the opposite angle).
//
// Read and written once, ~6 flops per element: bound by HBM.  A thread takes 16
// columns (two 16-byte pieces: eight pairs) of one token and up to four heads
// with the same cosines and sines, all their loads in flight at once.  A warp
// covers whole rows of consecutive tokens.  Calls back to back: 8192 tokens of 32
// heads, d = 128, 23.4 us (5.7 TB/s); one token of 32 sequences 4.0 to 4.7 us.
#include "fa_internal.h"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeLaunch a) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int TPR = D / 16;  // tasks per row
    const long long idx = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
    const int p = (int)(idx % TPR);
    const long long token = idx / TPR;
    if (token >= a.tokens) return;
    const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
    int c0, c1;
    task_columns<INTER>(p, a.rot, c0, c1);
    const bool turn = p < a.rot / 16;
    float c[8], s[8];
    if (turn) {
        const int pos = a.positions ? a.positions[token] : n;
        task_cos_sin(pos, a.turns + p * 8, a.magnitude, c, s);
        if (a.inverse)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
    const int h0 = blockIdx.y * a.hpt, h1 = min(h0 + a.hpt, a.H);
    const __nv_bfloat16* x = (const __nv_bfloat16*)a.x + b * a.xb + n * a.xn + h0 * a.xh;
    __nv_bfloat16* y = (__nv_bfloat16*)a.y + b * a.yb + n * a.yn + h0 * a.yh;
    constexpr int U = 4;
    for (int h = h0; h < h1; h += U, x += U * a.xh, y += U * a.yh) {
        uint4 u[U], w[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (h + i < h1) {
                u[i] = *reinterpret_cast<const uint4*>(x + i * a.xh + c0);
                w[i] = *reinterpret_cast<const uint4*>(x + i * a.xh + c1);
            }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (h + i < h1) {
                if (turn) rotate16<INTER>(u[i], w[i], c, s);
                *reinterpret_cast<uint4*>(y + i * a.yh + c0) = u[i];
                *reinterpret_cast<uint4*>(y + i * a.yh + c1) = w[i];
            }
    }
}

}  // namespace

cudaError_t launch_rope(RopeLaunch a, cudaStream_t s) {
    const long long blocks = (a.tokens * (a.d / 16) + kRopeThreads - 1) / kRopeThreads;
    // heads per thread: up to four share the sines while every SM still has four CTAs (8192 tokens of 32 heads, as
    // single graph replays: 1 head 55.3 us, 2 34.9, 4 26.7, 8 26.8)
    a.hpt = 4;
    while (a.hpt > 1 && blocks * ((a.H + a.hpt - 1) / a.hpt) < 4ll * a.num_sms) a.hpt /= 2;
    int groups = (a.H + a.hpt - 1) / a.hpt;
    if (groups > 65535) {
        a.hpt = (a.H + 65534) / 65535;
        groups = (a.H + a.hpt - 1) / a.hpt;
    }
    const dim3 grid((unsigned)blocks, (unsigned)groups), block(kRopeThreads);
    if (a.d == 128)
        return a.interleaved ? launch_dependent(rope_kernel<128, true>, grid, block, 0, s, a)
                             : launch_dependent(rope_kernel<128, false>, grid, block, 0, s, a);
    return a.interleaved ? launch_dependent(rope_kernel<64, true>, grid, block, 0, s, a)
                         : launch_dependent(rope_kernel<64, false>, grid, block, 0, s, a);
}

}  // namespace fa
