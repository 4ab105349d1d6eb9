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

// Every element is read once and written once.  Single tokens are bound by the latency of a launch and three dependent loads
// (length, table, token); prompts by latency too: each CTA has these loads, the sines and a barrier before its first store, and
// registers leave two of them on an SM (14 of 64 warps active).
//
// Measured, 8 kv heads, d = 128, rotated, with bounds: one token of 32 sequences 3.5 us; 8 ragged prompts of up to 2048 tokens
// 24.8 us (15.3 at HBM's copy rate; about 60% of DRAM's peak and half of the issue slots in a capture of 32 full ones).
//
// append_kernel: a CTA takes a run of tokens, in whole blocks, of up to four kv heads.  The tokens' places in the cache and
// their cosines and sines are made once, in shared memory; then each warp takes the keys of a head, or its values, for
// itself, without waiting for others: RP rows at a time, four of these loaded ahead, 16 columns of a row (the two pieces
// that a rotation pairs) per lane.  The extremes of a block gather in the lanes' registers over its rows and are joined by
// shuffles at its end.
//
// blocks_append_kernel is for blocks that are no multiple of RP rows (4, at d = 64 8): the rotated keys go to a tile in shared
// memory, and warps take the extremes from there.  (For blocks of any size, with two barriers per head, it took 26.8 us for
// 8 ragged prompts of up to 2048 tokens, 8 heads, d = 128, a third of the issue slots waiting for barriers.)
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

// The new tokens [t0, t1) of a unit that begins at token `first`; false if there are none.
struct AppendRun {
    int len, n, first, t0, t1;
};
__device__ __forceinline__ bool append_run(const PagedAppendLaunch& a, const PagedAppendPlan& plan, int b, int unit, AppendRun& r) {
    const int cap = a.max_pages * a.page, block = a.bounds ? a.block : 1;
    r.len = a.lens[b];
    r.n = a.new_lens ? a.new_lens[b] : a.N;
    if (r.len < 0 || r.len > cap || r.n < 0 || r.n > a.N || r.n > cap - r.len) {
        if (threadIdx.x == 0) record_invalid(a.err, kSiteCacheLen, r.len);
        r.len = min(max(r.len, 0), cap);
        r.n = min(min(max(r.n, 0), a.N), cap - r.len);
    }
    r.first = ((a.bounds ? (int)plan.block.div(r.len) : r.len) + unit * plan.unit) * block;
    r.t0 = max(r.len - r.first, 0);
    r.t1 = min(plan.unit * block, r.len + r.n - r.first);
    return r.n > 0 && r.first < r.len + r.n;
}

// Cosines and sines of `fresh` tokens, the first of which is new token `from`: [token][pair of pairs j < 4][task][2].  The
// positions are loaded for several tokens at once: one after the other the loads alone took 3 us.
__device__ __forceinline__ void make_turns(const PagedAppendLaunch& a, float2* s_turn, int turned, int b, int len, int from, int fresh) {
    const int q = threadIdx.x % 64, step = blockDim.x / 64;  // one pair for each of up to 64 threads, several tokens at a time
    if (q >= turned * 8) return;
    const uint64_t turns = a.turns[q];
    const int* positions = a.positions ? a.positions + (long long)b * a.N + from : nullptr;
    constexpr int AHEAD = 8;
    for (int t0 = threadIdx.x / 64; t0 < fresh; t0 += AHEAD * step) {
        int pos[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int tok = t0 + i * step;
            pos[i] = positions && tok < fresh ? positions[tok] : len + from + tok;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int tok = t0 + i * step;
            if (tok >= fresh) break;
            float2 cs;
            turn_cos_sin(pos[i], turns, a.magnitude, cs.x, cs.y);
            s_turn[((tok * 4 + q % 8 / 2) * turned + q / 8) * 2 + q % 2] = cs;
        }
    }
}
template <bool INTER>
__device__ __forceinline__ void turn_task(uint4& x, uint4& y, const float2* s_turn, int turned, int tok, int p) {
    const float2* cs = s_turn + (tok * 4 * turned + p) * 2;
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(cs + j * turned * 2);
        c[2 * j] = v.x, s[2 * j] = v.y, c[2 * j + 1] = v.z, s[2 * j + 1] = v.w;
    }
    rotate16<INTER>(x, y, c, s);
}

constexpr int kAppendWarps = 8, kMostTokens = 128;

// U: passes loaded ahead.
template <int D, int U, bool BOUNDS, bool INTER>
__global__ void __launch_bounds__(kAppendWarps * 32, 2) append_kernel(const PagedAppendLaunch a, const PagedAppendPlan plan) {
    extern __shared__ __align__(16) uint8_t s_mem[];
    __shared__ uint32_t s_row[kMostTokens], s_block[kMostTokens];  // places of the tokens' rows and of the blocks' bounds, head 0
    constexpr int TPR = D / 16, RP = 32 / TPR;
    pdl_launch_dependents();
    pdl_wait();
    const int group = blockIdx.x % plan.groups, unit = (blockIdx.x / plan.groups) % plan.units;
    const int b = blockIdx.x / plan.groups / plan.units, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    AppendRun run;
    if (!append_run(a, plan, b, unit, run)) return;
    const int block = BOUNDS ? a.block : 1, from = run.first + run.t0 - run.len, fresh = run.t1 - run.t0;
    const int turned = a.turns ? a.rot / 16 : 0;  // tasks of a row that rotate
    const float2* s_turn = reinterpret_cast<const float2*>(s_mem);
    // jobs: the keys of heads h0, h0 + 1, ..., then the values
    const int h0 = group * plan.heads, heads = min(plan.heads, a.Hkv - h0);
    const int r = lane / TPR, p = lane % TPR;
    int c0, c1;
    task_columns<INTER>(p, turned * 16, c0, c1);
    uint4 x[U], y[U];
    const int p0 = run.t0 / RP, p1 = (run.t1 + RP - 1) / RP;  // passes of RP tokens of the unit
    auto load_keys = [&](int h, int pass) {
        const __nv_bfloat16* src = (const __nv_bfloat16*)a.k + b * a.kb + h * a.kh;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = (pass + u) * RP + r;
            if (t >= run.t0 && t < run.t1) {
                const __nv_bfloat16* at = src + (long long)(from + t - run.t0) * a.kn;
                x[u] = *reinterpret_cast<const uint4*>(at + c0);
                y[u] = *reinterpret_cast<const uint4*>(at + c1);
            }
        }
    };
    if (warp < heads) load_keys(h0 + warp, p0);
    // the tokens' rows of the cache and the blocks' bounds
    for (int i = threadIdx.x; i < fresh; i += kAppendWarps * 32) {
        const int at = run.first + run.t0 + i, lpage = (int)plan.page.div(at), pg = a.table[(long long)b * a.max_pages + lpage];
        const bool ok = (unsigned)pg < (unsigned)a.num_pages;
        if (!ok) record_invalid(a.err, kSiteCacheTable, pg);
        s_row[i] = ok ? (uint32_t)pg * a.Hkv * a.page + (uint32_t)(at - lpage * a.page) : ~0u;
        if (BOUNDS) {
            const int blk = (int)plan.block.div(run.t0 + i);
            if (i == 0 || run.t0 + i == blk * block)
                s_block[blk] = ok ? (uint32_t)pg * a.Hkv * (a.page / block) + plan.block.div(at - lpage * a.page) : ~0u;
        }
    }
    if (turned) make_turns(a, reinterpret_cast<float2*>(s_mem), turned, b, run.len, from, fresh);
    __syncthreads();
    for (int job = warp; job < 2 * heads; job += kAppendWarps) {
        if (job >= heads) {  // values: whole rows, D / 8 lanes each
            constexpr int LPR = D / 8, RV = 32 / LPR, UV = 8;
            const int h = h0 + job - heads, vr = lane / LPR, c = lane % LPR * 8;
            const __nv_bfloat16* src = (const __nv_bfloat16*)a.v + b * a.vb + h * a.vh + (long long)(from + vr) * a.vn + c;
            for (int t = 0; t < fresh; t += UV * RV) {
                uint4 v[UV];
#pragma unroll
                for (int u = 0; u < UV; ++u)
                    if (t + u * RV + vr < fresh) v[u] = *reinterpret_cast<const uint4*>(src + (long long)(t + u * RV) * a.vn);
#pragma unroll
                for (int u = 0; u < UV; ++u) {
                    const uint32_t row = t + u * RV + vr < fresh ? s_row[t + u * RV + vr] : ~0u;
                    if (row != ~0u) *reinterpret_cast<uint4*>((__nv_bfloat16*)a.vp + (size_t)(row + h * a.page) * D + c) = v[u];
                }
            }
            continue;
        }
        const int h = h0 + job;
        if (job != warp) load_keys(h, p0);
        uint4 lo[2], hi[2], had = make_uint4(0, 0, 0, 0);
        // a block's bounds are four pieces per column pair: lanes r = 0 .. 3 have the smallest x, y and the largest x, y
        auto ends_at = [&](int blk) {
            const uint32_t row = s_block[blk];
            return row == ~0u || r > 3 ? nullptr
                                       : (__nv_bfloat16*)a.bounds + (size_t)(row + h * (a.page / block)) * (2 * D) +
                                             (r >= 2 ? D : 0) + (r & 1 ? c1 : c0);
        };
        const bool old = BOUNDS && run.len > run.first;  // the first block begins with earlier tokens
        if (old && ends_at(0)) had = *reinterpret_cast<const uint4*>(ends_at(0));
        bool begins = true;
        for (int pass = p0; pass < p1; pass += U) {
            uint4 u0[U], u1[U];
#pragma unroll
            for (int u = 0; u < U; ++u) u0[u] = x[u], u1[u] = y[u];
            if (pass + U < p1) load_keys(h, pass + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (pass + u >= p1) break;
                const int t = (pass + u) * RP + r, tok = t - run.t0;
                const bool there = t >= run.t0 && t < run.t1;
                if (there) {
                    if (p < turned) turn_task<INTER>(u0[u], u1[u], s_turn, turned, tok, p);
                    const uint32_t row = s_row[tok];
                    if (row != ~0u) {
                        __nv_bfloat16* dst = (__nv_bfloat16*)a.kp + (size_t)(row + h * a.page) * D;
                        *reinterpret_cast<uint4*>(dst + c0) = u0[u];
                        *reinterpret_cast<uint4*>(dst + c1) = u1[u];
                    }
                }
                if constexpr (BOUNDS) {
                    if (begins) {
                        lo[0] = lo[1] = make_uint4(0x7F807F80u, 0x7F807F80u, 0x7F807F80u, 0x7F807F80u);
                        hi[0] = hi[1] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
                    }
                    if (there) {
                        lo[0] = ends4(lo[0], u0[u], false), lo[1] = ends4(lo[1], u1[u], false);
                        hi[0] = ends4(hi[0], u0[u], true), hi[1] = ends4(hi[1], u1[u], true);
                    }
                    const int blk = (int)plan.block.div((pass + u) * RP);
                    begins = pass + u + 1 == p1 || (pass + u + 1) * RP == (blk + 1) * block;
                    if (begins) {  // the block's end
                        auto join = [&](uint4& v, bool is_max) {
#pragma unroll
                            for (int m = TPR; m < 32; m <<= 1)
                                v = ends4(v, make_uint4(__shfl_xor_sync(0xffffffffu, v.x, m), __shfl_xor_sync(0xffffffffu, v.y, m),
                                                        __shfl_xor_sync(0xffffffffu, v.z, m), __shfl_xor_sync(0xffffffffu, v.w, m)),
                                          is_max);
                        };
                        join(lo[0], false);
                        join(lo[1], false);
                        join(hi[0], true);
                        join(hi[1], true);
                        __nv_bfloat16* to = ends_at(blk);
                        if (to) {
                            uint4 v = r == 0 ? lo[0] : r == 1 ? lo[1] : r == 2 ? hi[0] : hi[1];
                            if (old && blk == 0) v = ends4(v, had, r >= 2);
                            *reinterpret_cast<uint4*>(to) = v;
                        }
                    }
                }
            }
        }
    }
}

template <int D, int HALF, int TPT, bool INTER>
__global__ void __launch_bounds__(2 * HALF, kPagedAppendThreads<TPT> / (2 * HALF))
    blocks_append_kernel(const PagedAppendLaunch a, const PagedAppendPlan plan) {
    extern __shared__ __align__(16) uint8_t s_mem[];
    constexpr int TPR = D / 16, WARPS = 2 * HALF / 32, STEP = HALF / TPR;  // STEP: tokens of one task per thread
    pdl_launch_dependents();
    pdl_wait();
    const int group = blockIdx.x % plan.groups;
    const int unit = (blockIdx.x / plan.groups) % plan.units;
    const int b = blockIdx.x / plan.groups / plan.units;
    const int is_v = threadIdx.x / HALF, tid = threadIdx.x % HALF, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    AppendRun run;
    if (!append_run(a, plan, b, unit, run)) return;
    const int block = a.block, len = run.len, first = run.first, t0 = run.t0, t1 = run.t1;
    const int fresh = t1 - t0, from = first + t0 - len;  // new tokens, the first one's index
    const int turned = a.turns ? a.rot / 16 : 0;  // tasks of a row that rotate
    float2* s_turn = reinterpret_cast<float2*>(s_mem);
    if (turned) {
        make_turns(a, s_turn, turned, b, len, from, fresh);
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
    const int blocks = (t1 + block - 1) / block, parts = blocks < WARPS ? WARPS / blocks : 1;
    __nv_bfloat16* ends[PER];
    {
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
        const bool old = warp == 0 && len > first && ends[0];  // the block that earlier tokens begin
        if (old) had = *reinterpret_cast<const uint4*>(ends[0]);
#pragma unroll
        for (int i = 0; i < TPT; ++i) x[i] = nx[i], y[i] = ny[i];
        if (h + 1 < h1) load();
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            if (!there[i]) continue;
            const int tok = tid / TPR + i * STEP;
            if (turn) turn_task<INTER>(x[i], y[i], s_turn, turned, tok, p);
            if (dst[i]) {
                *reinterpret_cast<uint4*>(dst[i]) = x[i];
                *reinterpret_cast<uint4*>(dst[i] + apart) = y[i];
                dst[i] += (long long)a.page * D;
            }
            if (!is_v) {
                *reinterpret_cast<uint4*>(s_tile + (tok * D + c0) * 2) = x[i];
                *reinterpret_cast<uint4*>(s_tile + (tok * D + c0 + apart) * 2) = y[i];
            }
        }
        {
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

template <int D, int HALF, int TPT, bool INTER>
cudaError_t launch_blocks_t(const PagedAppendLaunch& a, PagedAppendPlan plan, cudaStream_t s) {
    // kv heads per CTA, which share the sines: the fewest waves of resident CTAs times the work of one
    const long long cells = (long long)a.B * plan.units, slots = (long long)kPagedAppendThreads<TPT> / (2 * HALF) * a.num_sms;
    long long best = -1;
    for (int h = 8; h >= 1; h /= 2) {
        const long long waves = (cells * ((a.Hkv + h - 1) / h) + slots - 1) / slots, cost = waves * (2 * h + 3);
        if (best < 0 || cost < best) best = cost, plan.heads = h;
    }
    plan.groups = (a.Hkv + plan.heads - 1) / plan.heads;
    const int smem = plan.tokens * ((a.turns ? a.rot * 4 : 0) + D * 2) + std::max(kMostBlocks, 2 * HALF / 32) * D * 4;
    cudaError_t e = set_smem_limit_once<blocks_append_kernel<D, HALF, TPT, INTER>>(112 * 1024);
    if (e != cudaSuccess) return e;
    return launch_dependent(blocks_append_kernel<D, HALF, TPT, INTER>, dim3((unsigned)(cells * plan.groups)), dim3(2 * HALF),
                            (size_t)smem, s, a, plan);
}

template <int D, int HALF, int TPT>
cudaError_t launch_blocks(const PagedAppendLaunch& a, const PagedAppendPlan& plan, cudaStream_t s) {
    return a.interleaved ? launch_blocks_t<D, HALF, TPT, true>(a, plan, s) : launch_blocks_t<D, HALF, TPT, false>(a, plan, s);
}

template <int D, int U, bool BOUNDS, bool INTER>
cudaError_t launch_append(const PagedAppendLaunch& a, const PagedAppendPlan& plan, cudaStream_t s) {
    const int smem = a.turns ? plan.tokens * a.rot * 4 : 0;
    cudaError_t e = set_smem_limit_once<append_kernel<D, U, BOUNDS, INTER>>(64 * 1024);
    if (e != cudaSuccess) return e;
    return launch_dependent(append_kernel<D, U, BOUNDS, INTER>, dim3((unsigned)((long long)a.B * plan.units * plan.groups)),
                            dim3(kAppendWarps * 32), (size_t)smem, s, a, plan);
}

template <int D, int U>
cudaError_t launch_u(const PagedAppendLaunch& a, const PagedAppendPlan& plan, cudaStream_t s) {
    if (a.bounds)
        return a.interleaved ? launch_append<D, U, true, true>(a, plan, s) : launch_append<D, U, true, false>(a, plan, s);
    return a.interleaved ? launch_append<D, U, false, true>(a, plan, s) : launch_append<D, U, false, false>(a, plan, s);
}

template <int D>
cudaError_t launch_d(const PagedAppendLaunch& a, cudaStream_t s) {
    constexpr int RP = 512 / D;
    const bool rows = !a.bounds || a.block % RP == 0;  // blocks are whole passes of append_kernel
    const int block = a.bounds ? a.block : 1;
    const int touched = a.bounds ? (a.N + block - 2) / block + 1 : a.N;  // blocks that N tokens can touch
    PagedAppendPlan plan;
    plan.page = FastDiv((uint32_t)a.page);
    plan.block = FastDiv((uint32_t)block);
    auto units = [&](int tokens) {  // of whole blocks, about so many tokens each
        plan.unit = std::min(std::max(1, tokens / block), touched);
        plan.units = (touched + plan.unit - 1) / plan.unit;
        plan.tokens = std::min(plan.unit * block, a.N);
    };
    if (rows) {
        // four kv heads per CTA, a job for each warp (eight, which halve the sines: 26.6 us against 24.3 for 8 ragged prompts of
        // up to 2048 tokens, 8 heads, d = 128); 32 tokens, or 16 where that leaves SMs without two CTAs (16 sequences of up to
        // 200 tokens: 8.2 us with 32, 6.4 with 16); passes ahead: four (two: 26.1 us), for a few tokens two (32 single tokens
        // 3.9 us with four, 3.5 with two)
        plan.heads = 4;
        plan.groups = (a.Hkv + 3) / 4;
        units(32);
        if ((long long)a.B * plan.units * plan.groups < 2ll * a.num_sms) units(16);
        return a.N <= 2 * RP ? launch_u<D, 2>(a, plan, s) : launch_u<D, 4>(a, plan, s);
    }
    units(std::min(64, kMostBlocks * block));
    const int tasks = plan.tokens * (D / 16);
    if (tasks <= 128) return launch_blocks<D, 128, 1>(a, plan, s);
    if (tasks <= 256) return launch_blocks<D, 128, 2>(a, plan, s);
    if (tasks <= 512) return launch_blocks<D, 128, 4>(a, plan, s);
    return launch_blocks<D, 256, 4>(a, plan, s);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t s) {
    return a.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace fa
