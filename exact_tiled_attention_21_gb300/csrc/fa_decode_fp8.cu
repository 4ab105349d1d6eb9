// Attention of 1..16 new tokens per sequence over a paged cache held in 8 bits
// (e4m3 with one fp32 scale per block of sb tokens and kv head).
//
// Every byte of the cache is read once per 16 query rows (the Hq / Hkv heads of
// a group times the new tokens), 2 d bytes per key for 4 d flops per row: bound
// by HBM.  So each warp works alone.  It streams its own keys through a private
// ring of cp.async copies, in which every lane copies exactly the bytes that it
// will read as matrix fragments, so nothing waits for another warp until the
// warps' results are merged at the end.  One CTA (4 warps) takes a chunk of one
// (sequence, kv head, 16 rows).
//
// The products are mma.sync m16n8k16 with fp16 operands and fp32 sums, because
// an e4m3 value is exact in fp16 and the fragments can be read straight from
// the cache's rows: the order of d within Q K^T and of the keys within P V is
// free, so a lane's 16 consecutive bytes of a K row are the k-indices of its B
// fragments, and its 16 bytes of each of four V rows the k-pairs of its B
// fragments for d / 8 columns.  tcgen05 would need the bytes widened and written
// back to shared memory first (the queries are not 8 bits wide), and its 128
// rows are eight times what there is.
//
// q is scaled by a power of two per row into fp16's range (exact but for
// elements 2^-28 below the row's largest).  With x_j the score in log2 units,
// the softmax sums l = sum 2^(x_j - m) stay in fp32; the V product takes
// 2^(x_j + log2 vs_j - M) in fp16 (relative 2^-11, an eighth of the result's
// own bf16 step) with its own running maximum M, so that a block's scale can
// have any size.  Result: O 2^(M - m) / l.
#include "fa_e4m3.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
    static constexpr int KEYS = D == 128 ? 32 : 64;     // keys per warp and step (8 KB of K and V)
    static constexpr int STAGES = 3;                    // steps in flight
    static constexpr int HALF = KEYS * D;               // bytes of K (and of V) per step
    static constexpr int SLOT = 2 * HALF + 8 * KEYS;    // K, V, K scales, V scales
    static constexpr int RING = STAGES * SLOT;          // per warp
    static constexpr int OROW = D + 4;                  // row of the merge buffer, floats
    static constexpr int SMEM = kWarps * RING;
    static_assert(16 * OROW * 4 <= RING, "merge buffer");
    static_assert(kWarps * KEYS == (D == 128 ? kFp8ChunkKeys128 : kFp8ChunkKeys64), "chunk rule");
};

struct Params {
    const __nv_bfloat16* q;
    const uint8_t* kp;
    const uint8_t* vp;
    const float* ks;
    const float* vs;
    const int* table;
    const int* lens;
    __nv_bfloat16* o;
    float* lse;
    float* part_o;
    float* part_lse;
    float* scores;
    long long score_stride;
    int Hq, Hkv, Nq, max_pages, num_pages, splits, rows, row_tiles;
    uint32_t blocks_per_page;
    FastDiv page, sb;
    float scale_log2;
    DevError* err;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) decode_fp8_kernel(const Params a) {
    using C = Cfg<D>;
    constexpr int KEYS = C::KEYS, NT = KEYS / 8, KS = D / 16, DT = D / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_stat[kWarps][3][16];
    pdl_launch_dependents();
    pdl_wait();

    int idx = blockIdx.x;
    const int rt = idx % a.row_tiles; idx /= a.row_tiles;
    const int split = idx % a.splits; idx /= a.splits;
    const int kvh = idx % a.Hkv;
    const int b = idx / a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int P = (int)a.page.d, cap = a.max_pages * P;
    int len = a.lens[b];
    if (len < 0 || len > cap) {
        if (tid == 0) record_invalid(a.err, kSiteCacheLen, len);
        len = len < 0 ? 0 : cap;
    }
    constexpr int CHUNK = kWarps * KEYS;
    const int per = (len + a.splits - 1) / a.splits;
    const int chunk = (per + CHUNK - 1) / CHUNK * CHUNK;
    const int k0 = (int)min((long long)split * chunk, (long long)len), k1 = min(k0 + chunk, len);

    // rows of this tile, and the keys that each of this lane's two rows sees: j < lim
    const int r0 = rt * 16, nrows = min(16, a.rows - r0);
    const long long row0 = ((long long)b * a.Hq + (long long)kvh * (a.Hq / a.Hkv)) * a.Nq + r0;  // first row of the tile
    const int lim_lo = min(k1, len - a.Nq + (r0 + g) % a.Nq + 1), lim_hi = min(k1, len - a.Nq + (r0 + g + 8) % a.Nq + 1);

    // ---- Q fragments: k-step s of lane t is columns (D = 128: 64 (s / 4) +) 16 t + 4 (s % 4) .. + 3
    uint32_t qa[KS][4];
    float sc_lo, sc_hi;
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
        const int r = g + 8 * hi;
        uint32_t w[D / 8];  // D / 4 columns per lane
        if (r < nrows) {
            const uint4* src = reinterpret_cast<const uint4*>(a.q + (row0 + r) * D + t * 16);
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 x = src[i * 8 + j];
                    w[i * 8 + j * 4] = x.x, w[i * 8 + j * 4 + 1] = x.y, w[i * 8 + j * 4 + 2] = x.z,
                                  w[i * 8 + j * 4 + 3] = x.w;
                }
        } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) w[i] = 0;
        }
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // power of two that brings the row's largest element into [2^14, 2^15); rows of zeros, and of
        // infinities (which stay what they are), keep theirs
        int e = (int)(__float_as_uint(big) >> 23) - 127 - 14;
        if (big == 0.f || !(big <= 3.4e38f)) e = 0;
        e = max(e, -112);  // 2^-e stays a normal number
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        (hi ? sc_hi : sc_lo) = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t x = w[s * 2 + j];
                const __half2 h = __floats2half2_rn(__uint_as_float(x << 16) * down,
                                                    __uint_as_float(x & 0xFFFF0000u) * down);
                qa[s][hi + 2 * j] = *reinterpret_cast<const uint32_t*>(&h);
            }
    }

    // ---- the ring
    uint8_t* ring = smem + warp * C::RING;
    const uint32_t ring_u = smem_u32(ring);
    const int* trow = a.table + (long long)b * a.max_pages;
    const int first = k0 + warp * KEYS;                       // this warp's first key
    const int steps = first < k1 ? (k1 - first + CHUNK - 1) / CHUNK : 0;
    bool bad = false;
    int pg_next[KEYS / 32];  // pages of the next step's keys (one step ahead of their use)
    auto fetch_pages = [&](int it) {
#pragma unroll
        for (int i = 0; i < KEYS / 32; ++i) {
            const int key = first + it * CHUNK + i * 32 + lane;
            pg_next[i] = (it < steps && key < k1) ? trow[a.page.div(key)] : -1;
        }
    };
    auto issue = [&](int it, int slot) {
        if (it < steps) {
            const uint32_t base = ring_u + slot * C::SLOT;
            uint32_t row[KEYS / 32];  // cache row of key lane (+ 32), ~0 for none
#pragma unroll
            for (int i = 0; i < KEYS / 32; ++i) {
                const int key = first + it * CHUNK + i * 32 + lane;
                const int pg = pg_next[i];
                const bool in = key < k1, ok = in && (unsigned)pg < (unsigned)a.num_pages;
                bad |= in && !ok;
                const uint32_t at = (uint32_t)key - a.page.div(key) * P;
                const uint32_t head = (uint32_t)pg * a.Hkv + kvh;
                row[i] = ok ? head * P + at : ~0u;
                const uint32_t blk = ok ? head * a.blocks_per_page + a.sb.div(at) : 0u;
                const uint32_t dst = base + 2 * C::HALF + (i * 32 + lane) * 4;
                cp_async4(dst, a.ks + blk, ok);
                cp_async4(dst + 4 * KEYS, a.vs + blk, ok);
            }
            fetch_pages(it + 1);
            // K: lane (g, t) takes 16 bytes at 16 t (+ 64) of keys 8 j + g
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t rr = __shfl_sync(0xffffffffu, row[j / 4], (j % 4) * 8 + g);
                const uint8_t* src = a.kp + (size_t)(rr == ~0u ? 0u : rr) * D + t * 16;
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    cp_async16(base + ((j * (D / 64) + i) * 32 + lane) * 16, src + i * 64, rr != ~0u);
            }
            // V: lane (g, t) takes d / 8 bytes at g d / 8 of keys 16 i + 2 t, + 1, + 8, + 9
#pragma unroll
            for (int i = 0; i < KEYS / 16; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t rr =
                        __shfl_sync(0xffffffffu, row[i / 2], (i % 2) * 16 + 2 * t + (r & 1) + (r >> 1) * 8);
                    const uint8_t* src = a.vp + (size_t)(rr == ~0u ? 0u : rr) * D + g * DT;
                    const uint32_t dst = base + C::HALF + ((i * 4 + r) * 32 + lane) * DT;
                    if constexpr (D == 128)
                        cp_async16(dst, src, rr != ~0u);
                    else
                        cp_async8(dst, src, rr != ~0u);
                }
        }
        cp_async_commit();
    };

    float acc[DT][4];
#pragma unroll
    for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    float m_lo = -INFINITY, m_hi = -INFINITY, M_lo = -INFINITY, M_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;

    fetch_pages(0);
#pragma unroll
    for (int s = 0; s < C::STAGES; ++s) issue(s, s);
    int slot = 0;
    for (int it = 0; it < steps; ++it) {
        cp_async_wait<C::STAGES - 1>();
        __syncwarp();  // the scales were copied by other lanes
        const uint8_t* st = ring + slot * C::SLOT;
        const int key0 = first + it * CHUNK;
        float S[NT][4];
        const uint4* kf = reinterpret_cast<const uint4*>(st) + lane;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint4 x = kf[(j * (D / 64) + i) * 32];
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    mma_16816(S[j], qa[i * 4 + c], e4m3x2_to_half2(w[c]), e4m3x2_hi_to_half2(w[c]));
            }
        }
        const float2* ksf = reinterpret_cast<const float2*>(st + 2 * C::HALF);
        const float2* vsf = ksf + KEYS / 2;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float2 k2 = ksf[j * 4 + t];
            S[j][0] *= sc_lo * k2.x;
            S[j][1] *= sc_lo * k2.y;
            S[j][2] *= sc_hi * k2.x;
            S[j][3] *= sc_hi * k2.y;
        }
        if (key0 + KEYS > min(k1, len - a.Nq + 1)) {  // some row does not see every key
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int key = key0 + j * 8 + 2 * t;
                if (key >= lim_lo) S[j][0] = -INFINITY;
                if (key + 1 >= lim_lo) S[j][1] = -INFINITY;
                if (key >= lim_hi) S[j][2] = -INFINITY;
                if (key + 1 >= lim_hi) S[j][3] = -INFINITY;
            }
        }
        if (a.scores) {  // score_stride is even and covers every key, so a pair fits
            float* sr = a.scores + (row0 + g) * a.score_stride;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int key = key0 + j * 8 + 2 * t;
                if (key < k1) {
                    if (g < nrows) *reinterpret_cast<float2*>(sr + key) = make_float2(S[j][0], S[j][1]);
                    if (g + 8 < nrows)
                        *reinterpret_cast<float2*>(sr + 8 * a.score_stride + key) = make_float2(S[j][2], S[j][3]);
                }
            }
        }
        // ---- softmax: p = 2^(x - m) into l; w = 2^(x + log2 vs - M) for the value product
        float mx_lo = -INFINITY, mx_hi = -INFINITY;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            mx_lo = fmax3(mx_lo, S[j][0], S[j][1]);
            mx_hi = fmax3(mx_hi, S[j][2], S[j][3]);
        }
        mx_lo = fmaxf(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, 1));
        mx_hi = fmaxf(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, 1));
        mx_lo = fmaxf(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, 2));
        mx_hi = fmaxf(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, 2));
        const float mn_lo = fmaxf(m_lo, mx_lo), mn_hi = fmaxf(m_hi, mx_hi);
        const float b_lo = mn_lo == -INFINITY ? 0.f : mn_lo, b_hi = mn_hi == -INFINITY ? 0.f : mn_hi;
        l_lo *= ex2(m_lo - b_lo);
        l_hi *= ex2(m_hi - b_hi);
        m_lo = mn_lo;
        m_hi = mn_hi;
        float Mx_lo = -INFINITY, Mx_hi = -INFINITY;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float2 v2 = vsf[j * 4 + t];
            const float v0 = lg2(v2.x), v1 = lg2(v2.y);
            l_lo += ex2(S[j][0] - b_lo) + ex2(S[j][1] - b_lo);
            l_hi += ex2(S[j][2] - b_hi) + ex2(S[j][3] - b_hi);
            S[j][0] += v0;
            S[j][1] += v1;
            S[j][2] += v0;
            S[j][3] += v1;
            Mx_lo = fmax3(Mx_lo, S[j][0], S[j][1]);
            Mx_hi = fmax3(Mx_hi, S[j][2], S[j][3]);
        }
        Mx_lo = fmaxf(Mx_lo, __shfl_xor_sync(0xffffffffu, Mx_lo, 1));
        Mx_hi = fmaxf(Mx_hi, __shfl_xor_sync(0xffffffffu, Mx_hi, 1));
        Mx_lo = fmaxf(Mx_lo, __shfl_xor_sync(0xffffffffu, Mx_lo, 2));
        Mx_hi = fmaxf(Mx_hi, __shfl_xor_sync(0xffffffffu, Mx_hi, 2));
        if (__any_sync(0xffffffffu, Mx_lo > M_lo || Mx_hi > M_hi)) {
            const float n_lo = fmaxf(M_lo, Mx_lo), n_hi = fmaxf(M_hi, Mx_hi);
            const float f_lo = n_lo == -INFINITY ? 0.f : ex2(M_lo - n_lo), f_hi = n_hi == -INFINITY ? 0.f : ex2(M_hi - n_hi);
            M_lo = n_lo;
            M_hi = n_hi;
#pragma unroll
            for (int j = 0; j < DT; ++j) {
                acc[j][0] *= f_lo;
                acc[j][1] *= f_lo;
                acc[j][2] *= f_hi;
                acc[j][3] *= f_hi;
            }
        }
        const float B_lo = M_lo == -INFINITY ? 0.f : M_lo, B_hi = M_hi == -INFINITY ? 0.f : M_hi;
        const uint8_t* vf = st + C::HALF + lane * DT;
#pragma unroll
        for (int i = 0; i < KEYS / 16; ++i) {
            uint32_t pa[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float(&x)[4] = S[2 * i + h];
                const __half2 lo = __floats2half2_rn(ex2(x[0] - B_lo), ex2(x[1] - B_lo));
                const __half2 hi = __floats2half2_rn(ex2(x[2] - B_hi), ex2(x[3] - B_hi));
                pa[2 * h] = *reinterpret_cast<const uint32_t*>(&lo);
                pa[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&hi);
            }
            uint32_t v[4][DT / 4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(vf + (i * 4 + r) * 32 * DT);
                    v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(vf + (i * 4 + r) * 32 * DT);
                    v[r][0] = x.x, v[r][1] = x.y;
                }
            }
#pragma unroll
            for (int c = 0; c < DT / 4; ++c) {
                const uint32_t x0 = __byte_perm(v[0][c], v[1][c], 0x5140), y0 = __byte_perm(v[2][c], v[3][c], 0x5140);
                const uint32_t x1 = __byte_perm(v[0][c], v[1][c], 0x7362), y1 = __byte_perm(v[2][c], v[3][c], 0x7362);
                mma_16816(acc[4 * c], pa, e4m3x2_to_half2(x0), e4m3x2_to_half2(y0));
                mma_16816(acc[4 * c + 1], pa, e4m3x2_hi_to_half2(x0), e4m3x2_hi_to_half2(y0));
                mma_16816(acc[4 * c + 2], pa, e4m3x2_to_half2(x1), e4m3x2_to_half2(y1));
                mma_16816(acc[4 * c + 3], pa, e4m3x2_hi_to_half2(x1), e4m3x2_hi_to_half2(y1));
            }
        }
        __syncwarp();  // every lane has read the scales of this slot
        issue(it + C::STAGES, slot);
        slot = slot + 1 == C::STAGES ? 0 : slot + 1;
    }
    cp_async_wait<0>();
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_invalid(a.err, kSiteCacheTable, -1);

    // ---- merge the warps: O = sum_w O_w 2^(M_w - m) / l
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 1);
    l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 1);
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 2);
    l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 2);
    __syncwarp();
    if (t == 0) {
        s_stat[warp][0][g] = m_lo, s_stat[warp][0][g + 8] = m_hi;
        s_stat[warp][1][g] = l_lo, s_stat[warp][1][g + 8] = l_hi;
        s_stat[warp][2][g] = M_lo, s_stat[warp][2][g + 8] = M_hi;
    }
    float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int j = 0; j < DT; ++j) {
        mine[g * C::OROW + 2 * t * DT + j] = acc[j][0];
        mine[g * C::OROW + (2 * t + 1) * DT + j] = acc[j][1];
        mine[(g + 8) * C::OROW + 2 * t * DT + j] = acc[j][2];
        mine[(g + 8) * C::OROW + (2 * t + 1) * DT + j] = acc[j][3];
    }
    __syncthreads();
    for (int i = tid; i < nrows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_stat[w][0][r]);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += s_stat[w][1][r] * ex2(s_stat[w][0][r] - base);
        const float inv = l == 0.f ? 0.f : 1.f / l;  // 0: the row sees no key; NaN stays
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(smem + w * C::RING + (r * C::OROW + c) * 4);
            const float f = ex2(s_stat[w][2][r] - base) * inv;
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
        }
        const float lse2 = l == 0.f ? -INFINITY : m + lg2(l);
        if (a.splits == 1) {
            *reinterpret_cast<uint2*>(a.o + (row0 + r) * D + c) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
            if (a.lse && c == 0) a.lse[row0 + r] = lse2 * kLn2;
            if (a.scores && c == 0) a.part_lse[row0 + r] = lse2;
        } else {
            *reinterpret_cast<float4*>(a.part_o + ((row0 + r) * a.splits + split) * D + c) = o;
            if (c == 0) a.part_lse[(row0 + r) * a.splits + split] = lse2;
        }
    }
}

// ------------------------------------------------------------------ merge of the splits
// One warp per row: LSE = M + log2 sum 2^(lse_s - M), O = sum 2^(lse_s - LSE) o_s.  A split or row without
// keys has lse = -inf; a row without keys gets O = 0, LSE = -inf.
template <int D>
__global__ void __launch_bounds__(128) combine_fp8_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                                                          __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                                                          long long rows, int splits) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int PER = D / 32;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const float* pl = part_lse + row * splits;
    float M = -INFINITY;
    for (int s = lane; s < splits; s += 32) M = fmaxf(M, pl[s]);
    for (int w = 16; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    const float base = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
    for (int s = lane; s < splits; s += 32) sum += ex2(pl[s] - base);
    for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float out[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) out[i] = 0.f;
    const float* po = part_o + row * splits * D + lane * PER;
    for (int s = 0; s < splits; ++s) {
        const float w = ex2(pl[s] - base) * inv;
        if constexpr (PER == 4) {
            const float4 v = *reinterpret_cast<const float4*>(po + (long long)s * D);
            out[0] = fmaf(w, v.x, out[0]);
            out[1] = fmaf(w, v.y, out[1]);
            out[2] = fmaf(w, v.z, out[2]);
            out[3] = fmaf(w, v.w, out[3]);
        } else {
            const float2 v = *reinterpret_cast<const float2*>(po + (long long)s * D);
            out[0] = fmaf(w, v.x, out[0]);
            out[1] = fmaf(w, v.y, out[1]);
        }
    }
    __nv_bfloat16* ob = o + row * D + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; i += 2)
        *reinterpret_cast<__nv_bfloat162*>(ob + i) = __floats2bfloat162_rn(out[i], out[i + 1]);
    if (lse && lane == 0) lse[row] = sum == 0.f ? -INFINITY : (M + lg2(sum)) * kLn2;
}

// ------------------------------------------------------------------ accumulated weights
// weights[b, kvh, j] += sum over the group's rows of 2^(x_j - LSE), from the scores that the split kernel left.
// One thread takes four keys; the rows' LSEs come from the splits' partial ones.  Fixed order of additions.
constexpr int kWeightThreads = 128;
__global__ void __launch_bounds__(kWeightThreads) weights_fp8_kernel(const float* __restrict__ scores, long long stride,
                                                                     const float* __restrict__ part_lse,
                                                                     const int* __restrict__ lens,
                                                                     float* __restrict__ weights, int Hkv, int rows,
                                                                     int splits, int cap) {
    extern __shared__ float s_lse[];
    pdl_launch_dependents();
    pdl_wait();
    const int per_bh = (cap + kWeightThreads * 4 - 1) / (kWeightThreads * 4);
    const long long bh = blockIdx.x / per_bh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = min(max(lens[bh / Hkv], 0), cap);
    const int j0 = (int)(blockIdx.x % per_bh) * kWeightThreads * 4;
    if (j0 >= len) return;
    for (int r = warp; r < rows; r += kWeightThreads / 32) {
        const float* pl = part_lse + (bh * rows + r) * splits;
        float M = -INFINITY;
        for (int s = lane; s < splits; s += 32) M = fmaxf(M, pl[s]);
        for (int w = 16; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
        const float base = M == -INFINITY ? 0.f : M;
        float sum = 0.f;
        for (int s = lane; s < splits; s += 32) sum += ex2(pl[s] - base);
        for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        if (lane == 0) s_lse[r] = sum == 0.f ? INFINITY : M + lg2(sum);  // no keys: every weight 2^-inf = 0
    }
    __syncthreads();
    const int j = j0 + tid * 4;
    if (j >= len) return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* sr = scores + bh * rows * stride + j;
    for (int r = 0; r < rows; ++r, sr += stride) {
        const float4 x = *reinterpret_cast<const float4*>(sr);
        const float z = s_lse[r];
        sum.x += ex2(x.x - z);
        sum.y += ex2(x.y - z);
        sum.z += ex2(x.z - z);
        sum.w += ex2(x.w - z);
    }
    float* w = weights + bh * cap + j;
    w[0] += sum.x;
    if (j + 1 < len) w[1] += sum.y;
    if (j + 2 < len) w[2] += sum.z;
    if (j + 3 < len) w[3] += sum.w;
}

template <int D>
cudaError_t launch_d(const PagedDecodeFp8Launch& a, cudaStream_t s) {
    using C = Cfg<D>;
    cudaError_t e = set_smem_limit_once<decode_fp8_kernel<D>>(C::SMEM);
    if (e != cudaSuccess) return e;
    Params p;
    p.q = (const __nv_bfloat16*)a.q;
    p.kp = a.kp;
    p.vp = a.vp;
    p.ks = a.ks;
    p.vs = a.vs;
    p.table = a.table;
    p.lens = a.lens;
    p.o = (__nv_bfloat16*)a.o;
    p.lse = a.lse;
    p.part_o = a.part_o;
    p.part_lse = a.part_lse;
    p.scores = a.weights ? a.scores : nullptr;
    p.score_stride = a.score_stride;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.Nq = a.Nq;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.splits = a.splits;
    p.rows = a.Hq / a.Hkv * a.Nq;
    p.row_tiles = (p.rows + 15) / 16;
    p.blocks_per_page = (uint32_t)(a.page / a.sb);
    p.page = FastDiv((uint32_t)a.page);
    p.sb = FastDiv((uint32_t)a.sb);
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    const long long ctas = (long long)a.B * a.Hkv * a.splits * p.row_tiles;
    if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    e = launch_dependent(decode_fp8_kernel<D>, dim3((unsigned)ctas), dim3(kThreads), C::SMEM, s, p);
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.B * a.Hq * a.Nq;
    if (a.splits > 1) {
        e = launch_dependent(combine_fp8_kernel<D>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s,
                             (const float*)a.part_o, (const float*)a.part_lse, p.o, a.lse, rows, a.splits);
        if (e != cudaSuccess) return e;
    }
    if (!a.weights) return cudaSuccess;
    const int cap = a.max_pages * a.page;
    const long long blocks = (long long)((cap + kWeightThreads * 4 - 1) / (kWeightThreads * 4)) * a.B * a.Hkv;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    return launch_dependent(weights_fp8_kernel, dim3((unsigned)blocks), dim3(kWeightThreads), (size_t)p.rows * 4, s, (const float*)a.scores, a.score_stride,
                            (const float*)a.part_lse, a.lens, a.weights, a.Hkv, p.rows, a.splits, cap);
}

}  // namespace

cudaError_t launch_decode_paged_fp8(const PagedDecodeFp8Launch& a, cudaStream_t s) {
    return a.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

cudaError_t decode_fp8_blocks_per_sm(int d, int* blocks) {
    cudaError_t e = d == 128 ? set_smem_limit_once<decode_fp8_kernel<128>>(Cfg<128>::SMEM)
                             : set_smem_limit_once<decode_fp8_kernel<64>>(Cfg<64>::SMEM);
    if (e != cudaSuccess) return e;
    return d == 128 ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, decode_fp8_kernel<128>, kThreads, Cfg<128>::SMEM)
                    : cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, decode_fp8_kernel<64>, kThreads, Cfg<64>::SMEM);
}

}  // namespace fa
