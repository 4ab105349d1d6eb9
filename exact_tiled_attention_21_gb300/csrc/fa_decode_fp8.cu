// Attention of 1..16 new tokens per sequence over a paged cache held in 8 bits
// (e4m3 with one fp32 scale per block of sb tokens and kv head).
//
// Every byte of the cache is read once per 16 query rows (the Hq / Hkv heads of
// a group times the new tokens), 2 d bytes per key for 4 d flops per row: bound
// by HBM.  So each warp works alone.  It streams its own keys through a private
// ring of cp.async copies, so nothing waits for another warp until the warps'
// results are merged at the end.  One CTA (4 warps) takes a chunk of one
// (sequence, kv head, 16 rows).
//
// The products are mma.sync m16n8k16 with fp16 operands and fp32 sums, because
// an e4m3 value is exact in fp16 and the fragments can be read straight from
// the cache's rows.  Both are taken transposed, S^T = K Q^T and O^T = V^T P^T,
// so that the keys (and d) fill the 16 rows of a product and the queries its 8
// columns: up to 8 query rows cost half of what 16 do (NB = 1 or 2 column
// tiles).  The order of d within K Q^T and of the keys within V^T P^T is free: a
// lane's 16 consecutive bytes of a K row are the k-indices of its A fragments,
// and its d / 8 bytes of each of four V rows the k-pairs of its A fragments.  P
// turns from S^T's accumulators into the B fragments by an 8 x 8 transpose.
// tcgen05 would need the bytes widened and written back to shared memory first
// (the queries are not 8 bits wide), for 128-row products of at most 16 columns.
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
    static constexpr int STAGES = 2;                    // steps in flight
    static constexpr int HALF = KEYS * D;               // bytes of K (and of V) per step
    static constexpr int SLOT = 2 * HALF + 8 * KEYS;    // K, V, K scales, log2 of V scales
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

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, 3) decode_fp8_kernel(const Params a) {
    using C = Cfg<D>;
    constexpr int KEYS = C::KEYS, MT = KEYS / 16, KS = D / 16, DT = D / 8, ROWS = 8 * NB;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_stat[kWarps][3][ROWS];
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
    const int r0 = rt * ROWS, nrows = min(ROWS, a.rows - r0);  // query rows of this tile
    const long long row0 = ((long long)b * a.Hq + (long long)kvh * (a.Hq / a.Hkv)) * a.Nq + r0;

    // ---- the ring
    uint8_t* ring = smem + warp * C::RING;
    const uint32_t ring_u = smem_u32(ring);
    const int* trow = a.table + (long long)b * a.max_pages;
    const int first = k0 + warp * KEYS;                       // this warp's first key
    const int steps = first < k1 ? (k1 - first + CHUNK - 1) / CHUNK : 0;
    // A copy instruction moves whole rows (D / 16 lanes a row, so that a quarter warp asks for 128 consecutive bytes);
    // the fragments' readers find their 16 bytes (V at D = 64: 8) at
    //   K: (key / 8, half h of D = 128, lane' = 4 (key % 8) + t), lane' ^ 4 h
    //   V: (key / 16, r, 32-byte slot 4 s + (t ^ s), rest of the column), s = column / 32, at D = 64 t ^ s ^ 2 (r % 2),
    //   where key % 16 = 2 t + r % 2 + 8 (r / 2).
    // The exclusive-ors keep both the copies and the reads free of bank conflicts.  A 32-byte sector of a row stays
    // together: a copy whose sector is torn apart in shared memory fetches it from L2 once per piece (V in 16-byte
    // pieces: 1.5 times the bytes in all, which bound the kernel at 58 us of a 128k-token, 8-head cache).
    constexpr int LPR = D / 16, RPI = 32 / LPR;  // lanes per row, rows per copy instruction
    const int cr = lane / LPR, cc = lane % LPR;
    const uint8_t* kp = a.kp + cc * 16;
    const uint8_t* vp = a.vp + cc * 16;
    uint32_t kdst, vdst[2];  // this lane's slots (bytes) of the first copies
    if constexpr (D == 128) {
        kdst = ((cc >> 2) * 32 + ((4 * cr + (cc & 3)) ^ (cc & 4))) * 16;
        vdst[0] = C::HALF + ((cr & 1) * 16 + 4 * (cc >> 1) + ((cr >> 1) ^ (cc >> 1))) * 32 + (cc & 1) * 16;
        vdst[1] = vdst[0] ^ 64;  // t + 2
    } else {
        kdst = (4 * cr + cc) * 16;
        vdst[0] = C::HALF + ((cr & 1) * 8 + 4 * (cc >> 1) + ((cr >> 1) ^ ((cc >> 1) | (cr & 1) << 1))) * 32 + (cc & 1) * 16;
        vdst[1] = vdst[0] + 2 * 8 * 32;  // r + 2
    }
    bool bad = false;
    using Keys = int[KEYS / 32];     // of lane's key (+ 32) of a step
    using Scales = float[KEYS / 32];
    auto fetch_pages = [&](int it, Keys& pg) {
#pragma unroll
        for (int i = 0; i < KEYS / 32; ++i) {
            const int key = first + it * CHUNK + i * 32 + lane;
            pg[i] = (it < steps && key < k1) ? trow[a.page.div(key)] : -1;
        }
    };
    // Scales are loaded, not copied (a 4-byte copy asks L2 once per lane, a load once per sector), and put into the
    // ring one step later, when they have arrived; V's as logarithms.
    auto put_scales = [&](int slot, const Scales& ks, const Scales& vs) {
        float* f = reinterpret_cast<float*>(ring + slot * C::SLOT + 2 * C::HALF) + lane;
#pragma unroll
        for (int i = 0; i < KEYS / 32; ++i) {
            f[i * 32] = ks[i];
            f[KEYS + i * 32] = lg2(vs[i]);
        }
    };
    // ALL: every key of the step is there.
    auto copy = [&](uint32_t base, const uint32_t (&row)[KEYS / 32], const bool ALL) {
#pragma unroll
        for (int n = 0; n < KEYS / RPI; ++n) {
            const uint32_t rr = __shfl_sync(0xffffffffu, row[n * RPI / 32], (n * RPI + cr) & 31);
            const bool ok = ALL || rr != ~0u;
            const size_t off = (size_t)(ok ? rr : 0u) * D;
            uint32_t ko, vo;  // slots of copy n
            if constexpr (D == 128) {  // keys 4 n + cr
                ko = ((n >> 1) * 64 + (n & 1) * 16) * 16;
                vo = ((n >> 2) * 128 + ((n >> 1) & 1) * 64) * 16;
            } else {                   // keys 8 n + cr
                ko = n * 32 * 16;
                vo = (n >> 1) * 64 * 16;
            }
            cp_async16(base + kdst + ko, kp + off, ok);
            cp_async16(base + vdst[n & 1] + vo, vp + off, ok);
        }
    };
    auto issue = [&](int it, int slot, const Keys& pages, Scales& ks, Scales& vs) {
        if (it < steps) {
            uint32_t row[KEYS / 32];  // cache row of key lane (+ 32), ~0 for none
            bool all = true;
#pragma unroll
            for (int i = 0; i < KEYS / 32; ++i) {
                const int key = first + it * CHUNK + i * 32 + lane;
                const int pg = pages[i];
                const bool in = key < k1, ok = in && (unsigned)pg < (unsigned)a.num_pages;
                bad |= in && !ok;
                all &= ok;
                const uint32_t at = (uint32_t)key - a.page.div(key) * P;
                const uint32_t head = (uint32_t)pg * a.Hkv + kvh;
                row[i] = ok ? head * P + at : ~0u;
                const uint32_t blk = ok ? head * a.blocks_per_page + a.sb.div(at) : 0u;
                ks[i] = ok ? __ldg(a.ks + blk) : 0.f;
                vs[i] = ok ? __ldg(a.vs + blk) : 0.f;
            }
            if (__all_sync(0xffffffffu, all))
                copy(ring_u + slot * C::SLOT, row, true);
            else
                copy(ring_u + slot * C::SLOT, row, false);
        }
        cp_async_commit();
    };
    Keys pg_next;             // pages of the step after those in flight
    Scales ks_next, vs_next;  // scales of the step issued last
    {
        Keys pg[C::STAGES];
        Scales ks[C::STAGES], vs[C::STAGES];
#pragma unroll
        for (int s = 0; s < C::STAGES; ++s) fetch_pages(s, pg[s]);
        fetch_pages(C::STAGES, pg_next);
#pragma unroll
        for (int s = 0; s < C::STAGES; ++s) {
#pragma unroll
            for (int i = 0; i < KEYS / 32; ++i) ks[s][i] = vs[s][i] = 0.f;
            issue(s, s, pg[s], ks[s], vs[s]);
        }
#pragma unroll
        for (int s = 0; s + 1 < C::STAGES; ++s) put_scales(s, ks[s], vs[s]);
#pragma unroll
        for (int i = 0; i < KEYS / 32; ++i) {
            ks_next[i] = ks[C::STAGES - 1][i];
            vs_next[i] = vs[C::STAGES - 1][i];
        }
    }

    // ---- Q fragments: k-step s of lane (g, t) is row g, columns (D = 128: 64 (s / 4) +) 16 t + 4 (s % 4) .. + 3
    uint32_t qb[NB][KS][2];
    float sc[NB][2];  // score scale of the rows whose scores this lane holds: 8 nb + 2 t, + 1
    int lim[NB][2];   // and the keys that they see: j < lim
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        uint32_t w[D / 8];
        if (nb * 8 + g < nrows) {
            const uint4* src = reinterpret_cast<const uint4*>(a.q + (row0 + nb * 8 + g) * D + t * 16);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 x = src[i / 2 * 8 + i % 2];
                w[i * 4] = x.x, w[i * 4 + 1] = x.y, w[i * 4 + 2] = x.z, w[i * 4 + 3] = x.w;
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
        const float up = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t x = w[s * 2 + j];
                const __half2 h = __floats2half2_rn(__uint_as_float(x << 16) * down,
                                                    __uint_as_float(x & 0xFFFF0000u) * down);
                qb[nb][s][j] = *reinterpret_cast<const uint32_t*>(&h);
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            sc[nb][j] = __shfl_sync(0xffffffffu, up, (2 * t + j) * 4);
            lim[nb][j] = min(k1, len - a.Nq + (r0 + nb * 8 + 2 * t + j) % a.Nq + 1);
        }
    }

    float acc[D / 16][NB][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][nb][c] = 0.f;
    float m[NB][2], M[NB][2], l[NB][2];  // of rows 8 nb + 2 t + j
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) m[nb][j] = M[nb][j] = -INFINITY, l[nb][j] = 0.f;

    int slot = 0;
    for (int it = 0; it < steps; ++it) {
        put_scales(slot == 0 ? C::STAGES - 1 : slot - 1, ks_next, vs_next);
        cp_async_wait<C::STAGES - 1>();
        __syncwarp();  // every lane's copies are there
        const uint8_t* st = ring + slot * C::SLOT;
        const int key0 = first + it * CHUNK;
        float S[MT][NB][4];  // keys 16 i + g, + 8 (c / 2) of rows 8 nb + 2 t + c % 2
        const uint4* kf = reinterpret_cast<const uint4*>(st);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) S[i][nb][0] = S[i][nb][1] = S[i][nb][2] = S[i][nb][3] = 0.f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const int at = h * 32 + (lane ^ (4 * h));
                const uint4 x = kf[2 * i * (D / 64) * 32 + at], y = kf[(2 * i + 1) * (D / 64) * 32 + at];
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t ka[4] = {e4m3x2_to_half2(xw[c]), e4m3x2_to_half2(yw[c]), e4m3x2_hi_to_half2(xw[c]),
                                            e4m3x2_hi_to_half2(yw[c])};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma_16816(S[i][nb], ka, qb[nb][h * 4 + c][0], qb[nb][h * 4 + c][1]);
                }
            }
        }
        const float* ksf = reinterpret_cast<const float*>(st + 2 * C::HALF) + g;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float kscale = ksf[i * 16 + h * 8];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    S[i][nb][2 * h] *= sc[nb][0] * kscale;
                    S[i][nb][2 * h + 1] *= sc[nb][1] * kscale;
                }
            }
        if (key0 + KEYS > min(k1, len - a.Nq + 1)) {  // some row does not see every key
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (key0 + i * 16 + (c >> 1) * 8 + g >= lim[nb][c & 1]) S[i][nb][c] = -INFINITY;
        }
        if (a.scores) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float* sr = a.scores + (row0 + nb * 8 + 2 * t + j) * a.score_stride + key0 + g;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (nb * 8 + 2 * t + j < nrows && key0 + i * 16 + h * 8 + g < k1)
                                sr[i * 16 + h * 8] = S[i][nb][2 * h + j];
                }
        }
        // ---- softmax: p = 2^(x - m) into l; w = 2^(x + log2 vs - M) for the value product
        float base[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float mx = m[nb][j];
#pragma unroll
                for (int i = 0; i < MT; ++i) mx = fmax3(mx, S[i][nb][j], S[i][nb][2 + j]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                base[nb][j] = mx == -INFINITY ? 0.f : mx;
                l[nb][j] *= ex2(m[nb][j] - base[nb][j]);
                m[nb][j] = mx;
            }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float lv = ksf[KEYS + i * 16 + h * 8];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        l[nb][j] += ex2(S[i][nb][2 * h + j] - base[nb][j]);
                        S[i][nb][2 * h + j] += lv;
                    }
            }
        float Mx[NB][2];
        bool grown = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float mx = M[nb][j];
#pragma unroll
                for (int i = 0; i < MT; ++i) mx = fmax3(mx, S[i][nb][j], S[i][nb][2 + j]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                Mx[nb][j] = mx;
                grown |= mx > M[nb][j];
            }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float f[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f[j] = Mx[nb][j] == -INFINITY ? 0.f : ex2(M[nb][j] - Mx[nb][j]);
                    M[nb][j] = Mx[nb][j];
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[i][nb][c] *= f[c & 1];
            }
        }
        uint32_t pb[MT][NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const float b0 = M[nb][0] == -INFINITY ? 0.f : M[nb][0], b1 = M[nb][1] == -INFINITY ? 0.f : M[nb][1];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const __half2 w = __floats2half2_rn(ex2(S[i][nb][2 * h] - b0), ex2(S[i][nb][2 * h + 1] - b1));
                    pb[i][nb][h] = transpose8x8(*reinterpret_cast<const uint32_t*>(&w));
                }
        }
        const uint8_t* vf = st + C::HALF;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            uint32_t v[4][DT / 4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(vf + ((i * 4 + r) * 16 + 4 * (g >> 1) + (t ^ (g >> 1))) * 32 + (g & 1) * 16);
                    v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(
                        vf + ((i * 4 + r) * 8 + 4 * (g >> 2) + (t ^ ((g >> 2) | (r & 1) << 1))) * 32 + (g & 3) * 8);
                    v[r][0] = x.x, v[r][1] = x.y;
                }
            }
#pragma unroll
            for (int c = 0; c < DT / 4; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // columns g d / 8 + 4 c + 2 h (row g of the fragment) and + 1 (row g + 8)
                    const uint32_t sel = h ? 0x7362u : 0x5140u;
                    const uint32_t x = __byte_perm(v[0][c], v[1][c], sel), y = __byte_perm(v[2][c], v[3][c], sel);
                    const uint32_t va[4] = {e4m3x2_to_half2(x), e4m3x2_hi_to_half2(x), e4m3x2_to_half2(y),
                                            e4m3x2_hi_to_half2(y)};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma_16816(acc[2 * c + h][nb], va, pb[i][nb][0], pb[i][nb][1]);
                }
        }
        __syncwarp();  // every lane has read this slot
        issue(it + C::STAGES, slot, pg_next, ks_next, vs_next);
        fetch_pages(it + C::STAGES + 1, pg_next);
        slot = slot + 1 == C::STAGES ? 0 : slot + 1;
    }
    cp_async_wait<0>();
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_invalid(a.err, kSiteCacheTable, -1);

    // ---- merge the warps: O = sum_w O_w 2^(M_w - m) / l
    __syncwarp();
    float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = nb * 8 + 2 * t + j;
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], d);
            if (g == 0) s_stat[warp][0][r] = m[nb][j], s_stat[warp][1][r] = l[nb][j], s_stat[warp][2][r] = M[nb][j];
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                *reinterpret_cast<float2*>(mine + r * C::OROW + g * DT + 2 * i) =
                    make_float2(acc[i][nb][j], acc[i][nb][2 + j]);
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

template <int D, int NB>
cudaError_t launch_d(const PagedDecodeFp8Launch& a, cudaStream_t s) {
    using C = Cfg<D>;
    cudaError_t e = set_smem_limit_once<decode_fp8_kernel<D, NB>>(C::SMEM);
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
    p.row_tiles = (p.rows + 8 * NB - 1) / (8 * NB);
    p.blocks_per_page = (uint32_t)(a.page / a.sb);
    p.page = FastDiv((uint32_t)a.page);
    p.sb = FastDiv((uint32_t)a.sb);
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    const long long ctas = (long long)a.B * a.Hkv * a.splits * p.row_tiles;
    if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    e = launch_dependent(decode_fp8_kernel<D, NB>, dim3((unsigned)ctas), dim3(kThreads), C::SMEM, s, p);
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
    const bool one = a.Hq / a.Hkv * a.Nq <= 8;
    if (a.d == 128) return one ? launch_d<128, 1>(a, s) : launch_d<128, 2>(a, s);
    return one ? launch_d<64, 1>(a, s) : launch_d<64, 2>(a, s);
}

template <int D, int NB>
static cudaError_t blocks_per_sm(int* blocks) {
    const cudaError_t e = set_smem_limit_once<decode_fp8_kernel<D, NB>>(Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, decode_fp8_kernel<D, NB>, kThreads, Cfg<D>::SMEM);
}

cudaError_t decode_fp8_blocks_per_sm(int d, bool one, int* blocks) {
    if (d == 128) return one ? blocks_per_sm<128, 1>(blocks) : blocks_per_sm<128, 2>(blocks);
    return one ? blocks_per_sm<64, 1>(blocks) : blocks_per_sm<64, 2>(blocks);
}

}  // namespace fa
