// Writing new tokens into the paged bf16 cache, the keys rotated on the way,
// and keeping the bounds of each block's keys that a block selection reads.
//
// Layout: bf16 [num_pages, Hkv, page, d] for K and for V; bounds bf16
// [num_pages, Hkv, page / block, 2, d], the smallest and the largest element of
// each key column over the block's tokens.  Bounds are taken over the keys as
// they are stored, so they are exact; a NaN makes its column's bounds NaN.
#include <algorithm>

#include "fa_internal.h"
#include "fa_rope.cuh"

namespace fa {
namespace {

// One CTA per (sequence, run of blocks, run of kv heads); the first HALF threads take K, the others V.  Every element is
// read once and written once: bound by HBM for prompts, by the latency of a launch and three dependent loads (length,
// table, token) for single tokens.  A thread holds TPT tasks (16 columns of a token, the pieces that a rotation pairs) and
// loads the next head's while it works on this one's; the cosines and sines of the CTA's tokens are made once, in shared
// memory, and serve every head of the run.  For the bounds the rotated keys also go to a tile in shared memory: each warp
// takes the extremes over a part of a block's tokens, and one warp per block joins the parts with what the block had.
struct PagedAppendPlan {
    int unit, units, heads, groups;  // blocks per CTA (tokens without bounds), runs of them; kv heads per CTA, runs of them
    int tokens;                      // most new tokens of a CTA
    FastDiv page, block;
};

constexpr int kMostBlocks = 16;  // of a CTA

template <int TPT>
constexpr int kPagedAppendThreads = TPT > 2 ? 512 : TPT == 2 ? 768 : 1024;  // of an SM, by their registers

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint4 ends4(uint4 a, uint4 b, bool is_max) {
    return is_max ? make_uint4(max2(a.x, b.x), max2(a.y, b.y), max2(a.z, b.z), max2(a.w, b.w))
                  : make_uint4(min2(a.x, b.x), min2(a.y, b.y), min2(a.z, b.z), min2(a.w, b.w));
}

template <int D, int HALF, int TPT, bool BOUNDS, bool INTER>
__global__ void __launch_bounds__(2 * HALF, kPagedAppendThreads<TPT> / (2 * HALF))
    paged_append_kernel(const PagedAppendLaunch a, const PagedAppendPlan plan) {
    extern __shared__ __align__(16) uint8_t s_mem[];
    constexpr int TPR = D / 16, WARPS = 2 * HALF / 32, STEP = HALF / TPR;  // STEP: tokens of one task per thread
    pdl_launch_dependents();
    pdl_wait();
    const int group = blockIdx.x % plan.groups;
    const int unit = (blockIdx.x / plan.groups) % plan.units;
    const int b = blockIdx.x / plan.groups / plan.units;
    const int is_v = threadIdx.x / HALF, tid = threadIdx.x % HALF, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cap = a.max_pages * a.page, block = BOUNDS ? a.block : 1;
    int len = a.lens[b], n = a.new_lens ? a.new_lens[b] : a.N;
    if (len < 0 || len > cap || n < 0 || n > a.N || n > cap - len) {
        if (threadIdx.x == 0) record_invalid(a.err, kSiteCacheLen, len);
        len = min(max(len, 0), cap);
        n = min(min(max(n, 0), a.N), cap - len);
    }
    const int first = ((BOUNDS ? (int)plan.block.div(len) : len) + unit * plan.unit) * block;  // the CTA's first token
    if (n == 0 || first >= len + n) return;
    const int t0 = max(len - first, 0), t1 = min(plan.unit * block, len + n - first);  // its new tokens [t0, t1)
    const int fresh = t1 - t0, from = first + t0 - len;                                // their number, the first one's index
    const int turned = a.turns ? a.rot / 16 : 0;                                       // tasks of a row that rotate
    float2* s_turn = reinterpret_cast<float2*>(s_mem);                                 // [token][pair of pairs j < 4][task][2]
    if (turned) {
        const int q = threadIdx.x % 64;  // one pair for each of up to 64 threads, several tokens at a time
        if (q < turned * 8) {
            const uint64_t turns = a.turns[q];
            for (int tok = threadIdx.x / 64; tok < fresh; tok += 2 * HALF / 64) {
                const int pos = a.positions ? a.positions[(long long)b * a.N + from + tok] : len + from + tok;
                float2 cs;
                turn_cos_sin(pos, turns, a.magnitude, cs.x, cs.y);
                s_turn[((tok * 4 + q % 8 / 2) * turned + q / 8) * 2 + q % 2] = cs;
            }
        }
        __syncthreads();
    }
    // ---- the thread's tasks: the same columns of tokens tid / TPR, + STEP, ...
    const int h0 = group * plan.heads, h1 = min(h0 + plan.heads, a.Hkv), p = tid % TPR;
    const long long sn = is_v ? a.vn : a.kn, sh = is_v ? a.vh : a.kh;
    int c0, c1;
    task_columns<INTER>(p, is_v ? 0 : turned * 16, c0, c1);
    const int apart = c1 - c0;
    const bool turn = !is_v && p < turned;
    const __nv_bfloat16* src = (is_v ? (const __nv_bfloat16*)a.v + b * a.vb : (const __nv_bfloat16*)a.k + b * a.kb) +
                               (from + tid / TPR) * sn + h0 * sh + c0;
    __nv_bfloat16* dst[TPT];  // null: no such token, or no page for it
    bool there[TPT];
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const int tok = tid / TPR + i * STEP;
        there[i] = tok < fresh;
        dst[i] = nullptr;
        if (!there[i]) continue;
        const int at = first + t0 + tok, lpage = (int)plan.page.div(at);
        const int pg = a.table[(long long)b * a.max_pages + lpage];
        if ((unsigned)pg >= (unsigned)a.num_pages) {
            record_invalid(a.err, kSiteCacheTable, pg);
            continue;
        }
        dst[i] = (__nv_bfloat16*)(is_v ? a.vp : a.kp) +
                 (((long long)pg * a.Hkv + h0) * a.page + (at - lpage * a.page)) * D + c0;
    }
    uint4 nx[TPT], ny[TPT];  // the next head's
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < TPT; ++i)
            if (there[i]) {
                nx[i] = *reinterpret_cast<const uint4*>(src + i * STEP * sn);
                ny[i] = *reinterpret_cast<const uint4*>(src + i * STEP * sn + apart);
            }
        src += sh;
    };
    load();
    // ---- the blocks' bounds: a warp's blocks are warp, warp + WARPS
    uint8_t* s_tile = s_mem + (size_t)plan.tokens * turned * 64;
    uint4* s_part = reinterpret_cast<uint4*>(s_tile + (size_t)plan.tokens * D * 2);  // [item][2][D] bf16
    constexpr int LANES = D / 4, PER = (kMostBlocks + WARPS - 1) / WARPS;            // 16-byte pieces of a block's bounds
    const int blocks = BOUNDS ? (t1 + block - 1) / block : 0, parts = BOUNDS && blocks < WARPS ? WARPS / blocks : 1;
    __nv_bfloat16* ends[PER];
    if constexpr (BOUNDS) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int blk = warp + i * WARPS, at = first + blk * block, lpage = blk < blocks ? (int)plan.page.div(at) : 0;
            const int pg = blk < blocks ? a.table[(long long)b * a.max_pages + lpage] : -1;
            ends[i] = (unsigned)pg >= (unsigned)a.num_pages || lane >= LANES
                          ? nullptr
                          : (__nv_bfloat16*)a.bounds +
                                (((long long)pg * a.Hkv + h0) * plan.page.d + (at - lpage * a.page)) / block * (2 * D) + lane * 8;
        }
    }
    for (int h = h0; h < h1; ++h) {
        uint4 x[TPT], y[TPT], had;
        const bool old = BOUNDS && warp == 0 && len > first && ends[0];  // the block that earlier tokens begin
        if (old) had = *reinterpret_cast<const uint4*>(ends[0]);
#pragma unroll
        for (int i = 0; i < TPT; ++i) x[i] = nx[i], y[i] = ny[i];
        if (h + 1 < h1) load();
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            if (!there[i]) continue;
            const int tok = tid / TPR + i * STEP;
            if (turn) {
                const float2* cs = s_turn + (tok * 4 * turned + p) * 2;
                float c[8], s[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 v = *reinterpret_cast<const float4*>(cs + j * turned * 2);
                    c[2 * j] = v.x, s[2 * j] = v.y, c[2 * j + 1] = v.z, s[2 * j + 1] = v.w;
                }
                rotate16<INTER>(x[i], y[i], c, s);
            }
            if (dst[i]) {
                *reinterpret_cast<uint4*>(dst[i]) = x[i];
                *reinterpret_cast<uint4*>(dst[i] + apart) = y[i];
                dst[i] += (long long)a.page * D;
            }
            if (BOUNDS && !is_v) {
                *reinterpret_cast<uint4*>(s_tile + (tok * D + c0) * 2) = x[i];
                *reinterpret_cast<uint4*>(s_tile + (tok * D + c0 + apart) * 2) = y[i];
            }
        }
        if constexpr (BOUNDS) {
            __syncthreads();
            for (int it = warp; it < blocks * parts; it += WARPS) {
                const int blk = it / parts, part = it - blk * parts;
                const int s = max(blk * block, t0) - t0, e = min((blk + 1) * block, t1) - t0, per = (e - s + parts - 1) / parts;
                const int s1 = s + part * per, e1 = min(e, s1 + per);
                uint2 lo = make_uint2(0x7F807F80u, 0x7F807F80u), hi = make_uint2(0xFF80FF80u, 0xFF80FF80u);
                constexpr int RPW = 128 / D;  // rows of a warp's load, 4 columns per lane
#pragma unroll 4
                for (int r = s1 + lane / (D / 4); r < e1; r += RPW) {
                    const uint2 w = *reinterpret_cast<const uint2*>(s_tile + (r * D + lane % (D / 4) * 4) * 2);
                    lo.x = min2(lo.x, w.x), lo.y = min2(lo.y, w.y);
                    hi.x = max2(hi.x, w.x), hi.y = max2(hi.y, w.y);
                }
                if (RPW == 2) {
                    lo.x = min2(lo.x, __shfl_xor_sync(0xffffffffu, lo.x, 16));
                    lo.y = min2(lo.y, __shfl_xor_sync(0xffffffffu, lo.y, 16));
                    hi.x = max2(hi.x, __shfl_xor_sync(0xffffffffu, hi.x, 16));
                    hi.y = max2(hi.y, __shfl_xor_sync(0xffffffffu, hi.y, 16));
                }
                if (lane < D / 4) {
                    uint2* to = reinterpret_cast<uint2*>(s_part + it * LANES) + lane;
                    to[0] = lo;
                    to[D / 4] = hi;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int blk = warp + i * WARPS;
                if (blk >= blocks || !ends[i]) continue;
                const bool is_max = lane >= LANES / 2;
                uint4 v = s_part[blk * parts * LANES + lane];
                for (int part = 1; part < parts; ++part) v = ends4(v, s_part[(blk * parts + part) * LANES + lane], is_max);
                if (i == 0 && old) v = ends4(v, had, is_max);
                *reinterpret_cast<uint4*>(ends[i]) = v;
                ends[i] += (long long)(a.page / block) * (2 * D);
            }
        }
    }
}

template <int D, int HALF, int TPT, bool BOUNDS, bool INTER>
cudaError_t launch_t(const PagedAppendLaunch& a, PagedAppendPlan plan, cudaStream_t s) {
    // kv heads per CTA, which share the sines: the fewest waves of resident CTAs times the work of one
    const long long cells = (long long)a.B * plan.units, slots = (long long)kPagedAppendThreads<TPT> / (2 * HALF) * a.num_sms;
    long long best = -1;
    for (int h = 8; h >= 1; h /= 2) {
        const long long waves = (cells * ((a.Hkv + h - 1) / h) + slots - 1) / slots, cost = waves * (2 * h + 3);
        if (best < 0 || cost < best) best = cost, plan.heads = h;
    }
    plan.groups = (a.Hkv + plan.heads - 1) / plan.heads;
    const long long ctas = cells * plan.groups;
    const int smem = plan.tokens * ((a.turns ? a.rot * 4 : 0) + (BOUNDS ? D * 2 : 0)) +
                     (BOUNDS ? std::max(kMostBlocks, 2 * HALF / 32) * D * 4 : 0);
    cudaError_t e = set_smem_limit_once<paged_append_kernel<D, HALF, TPT, BOUNDS, INTER>>(112 * 1024);
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_append_kernel<D, HALF, TPT, BOUNDS, INTER>, dim3((unsigned)ctas), dim3(2 * HALF),
                            (size_t)smem, s, a, plan);
}

template <int D, int HALF, int TPT>
cudaError_t launch_ht(const PagedAppendLaunch& a, const PagedAppendPlan& plan, cudaStream_t s) {
    if (a.bounds)
        return a.interleaved ? launch_t<D, HALF, TPT, true, true>(a, plan, s) : launch_t<D, HALF, TPT, true, false>(a, plan, s);
    return a.interleaved ? launch_t<D, HALF, TPT, false, true>(a, plan, s) : launch_t<D, HALF, TPT, false, false>(a, plan, s);
}

template <int D>
cudaError_t launch_d(const PagedAppendLaunch& a, cudaStream_t s) {
    // a CTA's tokens: up to 64 (blocks of more than 64 tokens: one block), in whole blocks
    PagedAppendPlan plan;
    const int block = a.bounds ? a.block : 1;
    const int touched = a.bounds ? (a.N + block - 2) / block + 1 : a.N;  // blocks that N tokens can touch
    plan.unit = a.bounds ? std::min(std::max(1, std::min(64 / block, kMostBlocks)), touched) : std::min(64, a.N);
    plan.units = (touched + plan.unit - 1) / plan.unit;
    plan.tokens = std::min(plan.unit * block, a.N);
    plan.page = FastDiv((uint32_t)a.page);
    plan.block = FastDiv((uint32_t)block);
    const int tasks = plan.tokens * (D / 16);
    if (tasks <= 128) return launch_ht<D, 128, 1>(a, plan, s);
    if (tasks <= 256) return launch_ht<D, 128, 2>(a, plan, s);
    if (tasks <= 512) return launch_ht<D, 128, 4>(a, plan, s);
    return launch_ht<D, 256, 4>(a, plan, s);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t s) {
    return a.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace fa
