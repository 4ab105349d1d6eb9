// Attention of 1..16 new tokens per sequence over a paged cache held in 8 bits
// (e4m3 with one fp32 scale per block of sb tokens and kv head).
//
// Every byte of the cache is read once per 32 query rows (the Hq / Hkv heads of
// a group times the new tokens), 2 d bytes per key for 4 d flops per row: bound
// by HBM.  So each warp works alone: it streams its own keys through a private
// ring of cp.async copies, and nothing waits for another warp until the four
// warps' results of a CTA are merged.
//
// The work is one list of steps (128 keys at d = 128, 256 at d = 64) over all
// sequences, kv heads and row tiles, cut into equal shares for as many CTAs as
// run at once, from the lengths on the device: any batch of lengths, and any
// capacity of the block table, keeps every SM busy to the end.  A CTA's share
// crosses from one (sequence, kv head, row tile) to the next as it comes; the
// part of one that a CTA holds is a segment.  Segment results go to the
// workspace at slot CTA + item (which grows by one from each segment to the
// next) and a second kernel merges the segments of each row.
//
// The products are mma.sync m16n8k16 with fp16 operands and fp32 sums, because
// an e4m3 value is exact in fp16 and the fragments can be read straight from
// the cache's rows.  Both are taken transposed, S^T = K Q^T and O^T = V^T P^T,
// so that the keys (and d) fill the 16 rows of a product and the queries its 8
// columns: up to 8 query rows cost half of what 16 do (NB = 1, 2 or 4 column
// tiles).  The order of d within K Q^T and of the keys within V^T P^T is free: a
// lane's 16 consecutive bytes of a K row are the k-indices of its A fragments,
// and its d / 8 bytes of each of four V rows the k-pairs of its A fragments.  P
// turns from S^T's accumulators into the B fragments by an 8 x 8 transpose.
// tcgen05 would need the bytes widened and written back to shared memory first
// (the queries are not 8 bits wide), for 128-row products of at most 32 columns.
//
// q is scaled by a power of two per row into fp16's range (exact but for
// elements 2^-28 below the row's largest).  With x_j the score in log2 units,
// the softmax sums l = sum 2^(x_j - m) stay in fp32; the V product takes
// 2^(x_j + log2 vs_j - M) in fp16 (relative 2^-11, an eighth of the result's
// own bf16 step) with its own running maximum M, so that a block's scale can
// have any size.  Result: O 2^(M - m) / l.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "fa_e4m3.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr float kSlack = 8.f;  // how far (log2) a score may exceed the reference that its weight is relative to
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

template <int D, int NB>
struct Cfg {
    static constexpr int KEYS = D == 128 ? 32 : 64;     // keys per warp and step (8 KB of K and V)
    static constexpr int STEP = kWarps * KEYS;          // keys per CTA and step
    static constexpr int STAGES = 2;                    // steps in flight
    static constexpr int HALF = KEYS * D;               // bytes of K (and of V) per step
    static constexpr int SLOT = 2 * HALF + 8 * KEYS;    // K, V, K scales, log2 of V scales
    static constexpr int RING = STAGES * SLOT;          // per warp
    static constexpr int ROWS = 8 * NB;                 // query rows per tile
    static constexpr int OROW = D + 4;                  // row of a merge buffer, floats; within it column d (of 8 runs of
                                                        // D / 8: g, then 2 i + e) is at 16 i + 2 g + e: no bank conflicts
    static constexpr int BUFS = NB > 2 ? 2 : kWarps;    // merge buffers: one for each warp, or two in turns
    static constexpr int MERGE = kWarps * RING;         // byte offsets of the merge buffers
    static constexpr int QFRAGS = MERGE + BUFS * ROWS * OROW * 4;  // and of Q's fragments,
    static constexpr bool QSMEM = NB > 2;                          // which NB <= 2 has in registers
    static constexpr int SMEM = QFRAGS + (QSMEM ? ROWS * D * 2 : 0);
    // Registers: three CTAs' worth where that is enough.  Two run per SM: memory alone takes as long with one (128k
    // tokens: 51 us), and computing on top 68 us with one, 55 with two, 58 with three.
    static constexpr int REGS_FOR = NB > 1 ? 2 : 3, CTAS = 2;
    static_assert(CTAS * (SMEM + 2560) <= 227 * 1024, "shared memory");
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
    float* weights;
    float* part_o;       // [slot][ROWS][D], normalised
    float* part_lse;     // [slot][ROWS], log2
    float* scores;       // per (sequence, kv head) and tile [key][rows of the tile], log2; null without weights
    long long* prefix;   // [B + 1] steps before each sequence, per (kv head, row tile)
    int B, Hq, Hkv, Nq, max_pages, num_pages, rows, row_tiles, workers;
    uint32_t blocks_per_page;
    FastDiv page, sb;
    float scale_log2;
    DevError* err;
};

__device__ __forceinline__ int clamp_len(int len, int cap) { return min(max(len, 0), cap); }

// Steps of all sequences before q (64-bit warp scan of the lengths): the sequence that step q falls in, its first step
// and length.  With q beyond the end: sequence B and the total.  prefix: also written, if not null.
template <int STEP>
__device__ __forceinline__ void find_sequence(const int* lens, int B, int cap, long long q, long long* prefix, int& b,
                                              long long& start, int& len) {
    const int lane = threadIdx.x & 31;
    long long base = 0;
    b = B;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int l = b0 + lane < B ? clamp_len(lens[b0 + lane], cap) : 0;
        const uint32_t n = (uint32_t)(l + STEP - 1) / STEP;
        uint32_t incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
        if (prefix && b0 + lane < B) prefix[b0 + lane] = base + incl - n;
        const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > q);
        if (hit) {
            const int f = __ffs(hit) - 1;
            b = b0 + f;
            len = __shfl_sync(0xffffffffu, l, f);
            start = base + __shfl_sync(0xffffffffu, incl - n, f);
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    start = base;
    len = 0;
    if (prefix && lane == 0) prefix[B] = base;
}

// A position in the list of steps.
struct Cursor {
    int b, len, n;        // sequence, its length and steps
    int kvh, rt, s;       // kv head, row tile and step
};

template <int STEP>
__device__ __forceinline__ void advance(Cursor& c, const Params& a, int cap) {
    if (++c.s < c.n) return;
    c.s = 0;
    if (++c.rt < a.row_tiles) return;
    c.rt = 0;
    if (++c.kvh < a.Hkv) return;
    c.kvh = 0;
    do {
        ++c.b;
        c.len = c.b < a.B ? clamp_len(__ldg(a.lens + c.b), cap) : 0;
    } while (c.len == 0 && c.b < a.B);
    c.n = (c.len + STEP - 1) / STEP;
}

// Where the scores [key][rows of the tile] of a tile begin.  A (sequence, kv head)'s rows are padded to a multiple of
// four, so that a tile with a multiple of two or four rows has its scores of a key aligned to as many.
template <int ROWS>
__device__ __forceinline__ long long scores_at(const Params& a, long long bh, int rt, int cap) {
    return (bh * ((a.rows + 3) & ~3) + rt * ROWS) * cap;
}

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, Cfg<D, NB>::REGS_FOR) decode_fp8_kernel(const Params a) {
    using C = Cfg<D, NB>;
    constexpr int KEYS = C::KEYS, MT = KEYS / 16, KS = D / 16, DT = D / 8, ROWS = C::ROWS, STEP = C::STEP;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_stat[kWarps][2][ROWS];  // m and l
    __shared__ __align__(8) float s_up[ROWS];
    __shared__ Cursor s_ahead[kWarps];
    pdl_launch_dependents();
    pdl_wait();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int P = (int)a.page.d, cap = a.max_pages * P;
    if (blockIdx.x == 0)
        for (int i = tid; i < a.B; i += kThreads)
            if (a.lens[i] < 0 || a.lens[i] > cap) record_invalid(a.err, kSiteCacheLen, a.lens[i]);
    // this CTA's share [u, u1) of the steps
    const long long per_step = (long long)a.Hkv * a.row_tiles;
    long long u, u1;
    {
        int b, len;
        long long total;
        find_sequence<STEP>(a.lens, a.B, cap, LLONG_MAX, blockIdx.x == 0 && warp == 0 ? a.prefix : nullptr, b, total, len);
        total *= per_step;
        const long long workers = min((long long)a.workers, total);  // at least one step each
        if (blockIdx.x >= workers) return;
        u = blockIdx.x * total / workers;
        u1 = (blockIdx.x + 1ll) * total / workers;
    }
    Cursor cur;
    {
        long long start;
        find_sequence<STEP>(a.lens, a.B, cap, u / per_step, nullptr, cur.b, start, cur.len);
        cur.n = (cur.len + STEP - 1) / STEP;
        const long long in_b = u - start * per_step;
        const int item_b = (int)(in_b / cur.n);
        cur.s = (int)(in_b - (long long)item_b * cur.n);
        cur.kvh = item_b / a.row_tiles;
        cur.rt = item_b - cur.kvh * a.row_tiles;
    }
    const int count = (int)min(u1 - u, (long long)INT_MAX);  // steps (2^47 in all / workers; far below 2^31 in memory)

    // ---- the ring: this warp's keys of the steps ahead, whatever item they are of
    bool bad = false;
    uint8_t* ring = smem + warp * C::RING;
    const uint32_t ring_u = smem_u32(ring);
    uint2* qsm = reinterpret_cast<uint2*>(smem + C::QFRAGS);
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
    using Keys = int[KEYS / 32];     // of lane's key (+ 32) of a step
    using Scales = float[KEYS / 32];
    Cursor& ahead = s_ahead[warp];  // the step after those in `to_issue`; in shared memory to spare registers
    if (lane == 0) ahead = cur;
    __syncwarp();
    int fetched = 0, issued = 0;
    struct {
        Keys page;                 // pages of the lane's keys, loaded one step before their use
        int key0, len, kvh;
    } to_issue;
    auto fetch_pages = [&]() {
        to_issue.key0 = ahead.s * STEP + warp * KEYS;
        to_issue.len = ahead.len;
        to_issue.kvh = ahead.kvh;
        const int* trow = a.table + (long long)ahead.b * a.max_pages;
#pragma unroll
        for (int i = 0; i < KEYS / 32; ++i) {
            const int key = to_issue.key0 + i * 32 + lane;
            to_issue.page[i] = (fetched < count && key < ahead.len) ? trow[a.page.div(key)] : -1;
        }
        if (++fetched < count) {
            Cursor next = ahead;
            advance<STEP>(next, a, cap);
            __syncwarp();
            if (lane == 0) ahead = next;
            __syncwarp();
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
    auto issue = [&](int slot, Scales& ks, Scales& vs) {
        if (issued < count) {
            uint32_t row[KEYS / 32];  // cache row of key lane (+ 32), ~0 for none
            bool all = true;
#pragma unroll
            for (int i = 0; i < KEYS / 32; ++i) {
                const int key = to_issue.key0 + i * 32 + lane;
                const int pg = to_issue.page[i];
                const bool in = key < to_issue.len, ok = in && (unsigned)pg < (unsigned)a.num_pages;
                bad |= in && !ok;
                all &= ok;
                const uint32_t at = (uint32_t)key - a.page.div(key) * P;
                const uint32_t head = (uint32_t)pg * a.Hkv + to_issue.kvh;
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
        ++issued;
        cp_async_commit();
    };
    Scales ks_next, vs_next;  // scales of the step issued last
    static_assert(C::STAGES == 2, "the start below");
    {
        Scales ks, vs;
        fetch_pages();
        auto first = to_issue;
        fetch_pages();
        auto second = to_issue;
        fetch_pages();
        const auto third = to_issue;
        to_issue = first;
#pragma unroll
        for (int i = 0; i < KEYS / 32; ++i) ks[i] = vs[i] = ks_next[i] = vs_next[i] = 0.f;
        issue(0, ks, vs);
        to_issue = second;
        issue(1, ks_next, vs_next);
        to_issue = third;
        put_scales(0, ks, vs);
    }

    // ---- what a segment holds
    uint32_t qb[C::QSMEM ? 1 : NB][KS][2];
    float sc[C::QSMEM ? 1 : NB][2];  // (NB <= 2) score scale of the rows whose scores this lane holds: 8 nb + 2 t, + 1
    float acc[D / 16][NB][4];
    float m[NB][2], M[NB][2], l[NB][2];  // of rows 8 nb + 2 t + j; the maxima start at the lowest number: a row
                                         // that sees no key keeps l = 0 (2^(-inf - m))
    int seg = 0;  // first step of the segment within its item
    bool begins = true;
    int slot = 0;
    for (int it = 0; it < count; ++it) {
    const int r0 = cur.rt * ROWS, nrows = min(ROWS, a.rows - r0);      // query rows of the tile
    const long long bh = (long long)cur.b * a.Hkv + cur.kvh;
    const long long row0 = bh * a.rows + r0;                           // (b, head, token) flattened
    if (begins) {
    seg = cur.s;
    // ---- Q fragments: k-step s of lane (g, t) is row g, columns (D = 128: 64 (s / 4) +) 16 t + 4 (s % 4) .. + 3
#pragma unroll
    for (int f = 0; f < (C::QSMEM ? 1 : NB); ++f) {
        const int nb = C::QSMEM ? warp : f;  // in shared memory each warp makes one column tile
        static_assert(!C::QSMEM || NB == kWarps, "one column tile per warp");
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
        for (int s = 0; s < KS; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t x = w[s * 2 + j];
                const __half2 h = __floats2half2_rn(__uint_as_float(x << 16) * down,
                                                    __uint_as_float(x & 0xFFFF0000u) * down);
                qb[f][s][j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if constexpr (C::QSMEM) qsm[(s * NB + nb) * 32 + lane] = make_uint2(qb[0][s][0], qb[0][s][1]);
        }
        if constexpr (C::QSMEM) {
            if (t == 0) s_up[nb * 8 + g] = up;
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) sc[f][j] = __shfl_sync(0xffffffffu, up, (2 * t + j) * 4);
        }
    }
    if constexpr (C::QSMEM) {
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][nb][c] = 0.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) m[nb][j] = M[nb][j] = -FLT_MAX, l[nb][j] = 0.f;
    }

    const int key0 = cur.s * STEP + warp * KEYS;
        cp_async_wait<C::STAGES - 1>();
        __syncwarp();  // every lane's copies are there
        const uint8_t* st = ring + slot * C::SLOT;
        if (key0 < cur.len) {
        float S[MT][NB][4];  // keys 16 i + g, + 8 (c / 2) of rows 8 nb + 2 t + c % 2
        const uint4* kf = reinterpret_cast<const uint4*>(st);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) S[i][nb][0] = S[i][nb][1] = S[i][nb][2] = S[i][nb][3] = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            uint32_t w[2 * MT][4];
            const int at = h * 32 + (lane ^ (4 * h));
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                const uint4 x = kf[i * (D / 64) * 32 + at];
                w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t q0[NB], q1[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if constexpr (C::QSMEM) {
                        const uint2 x = qsm[((h * 4 + c) * NB + nb) * 32 + lane];
                        q0[nb] = x.x, q1[nb] = x.y;
                    } else {
                        q0[nb] = qb[nb][h * 4 + c][0], q1[nb] = qb[nb][h * 4 + c][1];
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint32_t ka[4] = {e4m3x2_to_half2(w[2 * i][c]), e4m3x2_to_half2(w[2 * i + 1][c]),
                                            e4m3x2_hi_to_half2(w[2 * i][c]), e4m3x2_hi_to_half2(w[2 * i + 1][c])};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma_16816(S[i][nb], ka, q0[nb], q1[nb]);
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
                    float2 x;
                    if constexpr (C::QSMEM)
                        x = *reinterpret_cast<const float2*>(s_up + nb * 8 + 2 * t);
                    else
                        x = make_float2(sc[nb][0], sc[nb][1]);
                    S[i][nb][2 * h] *= x.x * kscale;
                    S[i][nb][2 * h + 1] *= x.y * kscale;
                }
            }
        if (key0 + MT * 16 > cur.len - a.Nq + 1) {  // some row does not see every key
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int lim = cur.len - a.Nq + (r0 + nb * 8 + 2 * t + j) % a.Nq + 1 - key0 - g;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (i * 16 + h * 8 >= lim) S[i][nb][2 * h + j] = -INFINITY;
                }
        }
        if (a.scores) {  // [key][row of the tile]: a lane's two rows are neighbours
            float* sr = a.scores + scores_at<ROWS>(a, bh, cur.rt, cap) + (long long)(key0 + g) * nrows + 2 * t;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (key0 + i * 16 + h * 8 + g < cur.len)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            float* at = sr + (i * 16 + h * 8) * nrows + nb * 8;
                            if ((nrows & 1) == 0) {
                                if (nb * 8 + 2 * t < nrows)
                                    *reinterpret_cast<float2*>(at) = make_float2(S[i][nb][2 * h], S[i][nb][2 * h + 1]);
                            } else {
                                if (nb * 8 + 2 * t < nrows) at[0] = S[i][nb][2 * h];
                                if (nb * 8 + 2 * t + 1 < nrows) at[1] = S[i][nb][2 * h + 1];
                            }
                        }
        }
        // ---- softmax: p = 2^(x - m) into l; w = 2^(x + log2 vs - M) for the value product.  m and M need not be the
        // maxima, only within 2^8 of them (fp16 holds 2^15): most steps find no larger one and skip the reductions.
        float mx[NB][2];
        bool grown = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mx[nb][j] = fmaxf(S[0][nb][j], S[0][nb][2 + j]);
#pragma unroll
                for (int i = 1; i < MT; ++i) mx[nb][j] = fmax3(mx[nb][j], S[i][nb][j], S[i][nb][2 + j]);
                grown |= mx[nb][j] > m[nb][j] + kSlack;
            }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(m[nb][j], mx[nb][j]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    l[nb][j] *= ex2(m[nb][j] - x);
                    m[nb][j] = x;
                }
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
                        l[nb][j] += ex2(S[i][nb][2 * h + j] - m[nb][j]);
                        S[i][nb][2 * h + j] += lv;
                    }
            }
        grown = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mx[nb][j] = fmaxf(S[0][nb][j], S[0][nb][2 + j]);
#pragma unroll
                for (int i = 1; i < MT; ++i) mx[nb][j] = fmax3(mx[nb][j], S[i][nb][j], S[i][nb][2 + j]);
                grown |= mx[nb][j] > M[nb][j] + kSlack;
            }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(M[nb][j], mx[nb][j]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    const float f = ex2(M[nb][j] - x);
                    M[nb][j] = x;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        acc[i][nb][j] *= f;
                        acc[i][nb][2 + j] *= f;
                    }
                }
        }
        uint32_t pb[MT][NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const __half2 w = __floats2half2_rn(ex2(S[i][nb][2 * h] - M[nb][0]),
                                                        ex2(S[i][nb][2 * h + 1] - M[nb][1]));
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
        }
        put_scales(slot ^ 1, ks_next, vs_next);
        __syncwarp();  // every lane has read this slot
        issue(slot, ks_next, vs_next);
        fetch_pages();
        slot ^= 1;

    // ---- at the segment's end, merge the warps: O = sum_w O_w 2^(M_w - m) / l
    const bool item_ends = cur.s + 1 == cur.n;
    begins = item_ends || it + 1 == count;
    if (begins) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = nb * 8 + 2 * t + j;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], d);
                if (g == 0) s_stat[warp][0][r] = m[nb][j], s_stat[warp][1][r] = l[nb][j];
            }
        __syncthreads();
        float f[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = nb * 8 + 2 * t + j;
                float top = s_stat[0][0][r];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_stat[w][0][r]);
                f[nb][j] = ex2(M[nb][j] - top);
            }
        float* buf = reinterpret_cast<float*>(smem + C::MERGE) + (warp % C::BUFS) * ROWS * C::OROW;
#pragma unroll 1
        for (int turn = 0; turn < kWarps / C::BUFS; ++turn) {
            if (warp / C::BUFS == turn) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            float2* at = reinterpret_cast<float2*>(buf + (nb * 8 + 2 * t + j) * C::OROW + i * 16 + g * 2);
                            float2 x = make_float2(acc[i][nb][j] * f[nb][j], acc[i][nb][2 + j] * f[nb][j]);
                            if (turn) {
                                const float2 y = *at;
                                x.x += y.x;
                                x.y += y.y;
                            }
                            *at = x;
                        }
            }
            __syncthreads();
        }
        const bool whole = seg == 0 && item_ends;
        const long long slot_out = blockIdx.x + bh * a.row_tiles + cur.rt;
        for (int i = tid; i < nrows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i % (D / 4)) * 4, at = c % DT * 8 + c / DT * 2;
            float top = s_stat[0][0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_stat[w][0][r]);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_stat[w][1][r] * ex2(s_stat[w][0][r] - top);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // 0: the row sees no key; NaN stays
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::BUFS; ++w) {
                const float* x = reinterpret_cast<const float*>(smem + C::MERGE) + (w * ROWS + r) * C::OROW + at;
                o.x += x[0];
                o.y += x[1];
                o.z += x[16];
                o.w += x[17];
            }
            o.x *= inv;
            o.y *= inv;
            o.z *= inv;
            o.w *= inv;
            const float lse2 = sum == 0.f ? -INFINITY : top + lg2(sum);
            if (whole) {
                *reinterpret_cast<uint2*>(a.o + (row0 + r) * D + c) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
                if (a.lse && c == 0) a.lse[row0 + r] = lse2 * kLn2;
            } else {
                *reinterpret_cast<float4*>(a.part_o + (slot_out * ROWS + r) * D + c) = o;
            }
            if (c == 0) a.part_lse[slot_out * ROWS + r] = lse2;
        }
        __syncthreads();  // the buffers and Q are the next segment's
    }
    if (it + 1 < count) advance<STEP>(cur, a, cap);
    }
    cp_async_wait<0>();
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_invalid(a.err, kSiteCacheTable, -1);
}

// ------------------------------------------------------------------ merge of the segments, and the weights
// The segments of item i (sequence b, kv head, row tile) are those of the CTAs that hold its first to its last step;
// CTA c's is in slot c + i.  Returns their number (0: an empty sequence) and the first one's slot.
__device__ __forceinline__ int find_segments(const Params& a, int b, int item_b, long long& slot) {
    const long long per_step = (long long)a.Hkv * a.row_tiles;
    const long long p0 = a.prefix[b], n = a.prefix[b + 1] - p0, total = a.prefix[a.B] * per_step;
    if (n == 0) return 0;
    const long long s0 = p0 * per_step + item_b * n, s1 = s0 + n - 1;  // first and last step
    const long long workers = min((long long)a.workers, total);
    const long long c0 = ((s0 + 1) * workers - 1) / total, c1 = ((s1 + 1) * workers - 1) / total;
    slot = c0 + b * per_step + item_b;
    return (int)(c1 - c0) + 1;
}

// log2-domain LSE of a row over its segments, by one warp; M: the largest partial one (0 for none).  +inf sum: NaN stays.
__device__ __forceinline__ float merge_lse(const float* pl, int stride, int segs, float& base) {
    const int lane = threadIdx.x & 31;
    float M = -INFINITY;
    for (int s = lane; s < segs; s += 32) M = fmaxf(M, pl[(long long)s * stride]);
    for (int w = 16; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    base = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
    for (int s = lane; s < segs; s += 32) sum += ex2(pl[(long long)s * stride] - base);
    for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    return sum;
}

constexpr int kFinishThreads = 128, kWeightTokens = 4;  // tokens per thread of the weights

// Blocks below `row_blocks`: one row each; LSE = M + log2 sum 2^(lse_s - M), O = sum 2^(lse_s - M) o_s / sum, the
// segments dealt to groups of D / 4 threads.  A row without keys gets O = 0, LSE = -inf; a row whose item was one
// segment is already written.
// The others, with weights: 512 tokens of one (sequence, kv head) each; weights[j] += sum over the rows of
// 2^(x_j - LSE), one thread per token, in a fixed order.
template <int D, int ROWS>
__global__ void __launch_bounds__(kFinishThreads) finish_fp8_kernel(const Params a, unsigned row_blocks, int weight_blocks) {
    constexpr int LANES = D / 4, GROUPS = kFinishThreads / LANES, AHEAD = 4;
    extern __shared__ float s_lse[];  // weights: LSE of the rows
    __shared__ float4 s_o[GROUPS][LANES];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x;
    if (blockIdx.x < row_blocks) {
        const long long row = blockIdx.x, bh = row / a.rows;
        const int r = (int)(row - bh * a.rows), b = (int)(bh / a.Hkv), rt = r / ROWS;
        long long slot = 0;
        const int segs = find_segments(a, b, (int)(bh % a.Hkv) * a.row_tiles + rt, slot);
        if (segs == 1) return;
        const int grp = tid / LANES, col = tid % LANES;
        const long long at = slot * ROWS + (r - rt * ROWS);
        const float* pl = a.part_lse + at;
        const float4* po = reinterpret_cast<const float4*>(a.part_o + at * D) + col;
        float4 v[AHEAD];  // the first segments, loaded before the weights are known
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (grp + i * GROUPS < segs) v[i] = po[(long long)(grp + i * GROUPS) * ROWS * LANES];
        float base;
        const float sum = merge_lse(pl, ROWS, segs, base);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = grp; s0 < segs; s0 += AHEAD * GROUPS) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int s = s0 + i * GROUPS;
                if (s < segs) {
                    const float w = ex2(pl[(long long)s * ROWS] - base) * inv;
                    o.x = fmaf(w, v[i].x, o.x);
                    o.y = fmaf(w, v[i].y, o.y);
                    o.z = fmaf(w, v[i].z, o.z);
                    o.w = fmaf(w, v[i].w, o.w);
                }
                if (s + AHEAD * GROUPS < segs) v[i] = po[(long long)(s + AHEAD * GROUPS) * ROWS * LANES];
            }
        }
        s_o[grp][col] = o;
        __syncthreads();
        if (grp == 0) {
#pragma unroll
            for (int i = 1; i < GROUPS; ++i) {
                const float4 x = s_o[i][col];
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
            }
            *reinterpret_cast<uint2*>(a.o + row * D + col * 4) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
            if (a.lse && col == 0) a.lse[row] = sum == 0.f ? -INFINITY : (base + lg2(sum)) * kLn2;
        }
        return;
    }
    const unsigned idx = blockIdx.x - row_blocks;
    const long long bh = idx / weight_blocks;
    const int b = (int)(bh / a.Hkv), kvh = (int)(bh % a.Hkv), cap = a.max_pages * (int)a.page.d;
    const int len = clamp_len(a.lens[b], cap), j0 = (int)(idx % weight_blocks) * kFinishThreads * kWeightTokens;
    if (j0 >= len) return;
    // the rows' LSEs, a tile at a time: kFinishThreads / ROWS lanes per row
    constexpr int LPR = kFinishThreads / ROWS;
    for (int rt = 0; rt < a.row_tiles; ++rt) {
        long long slot = 0;
        const int segs = find_segments(a, b, kvh * a.row_tiles + rt, slot);
        const int r = tid / LPR;
        const float* pl = a.part_lse + slot * ROWS + r;
        const bool row = rt * ROWS + r < a.rows;
        float M = -FLT_MAX, sum = 0.f;
        for (int s = tid % LPR; row && s < segs; s += LPR) M = fmaxf(M, pl[(long long)s * ROWS]);
#pragma unroll
        for (int w = LPR / 2; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
        for (int s = tid % LPR; row && s < segs; s += LPR) sum += ex2(pl[(long long)s * ROWS] - M);
#pragma unroll
        for (int w = LPR / 2; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        if (row && tid % LPR == 0) s_lse[rt * ROWS + r] = sum == 0.f ? INFINITY : M + lg2(sum);  // no keys: 2^-inf = 0
    }
    __syncthreads();
    float sum[kWeightTokens], before[kWeightTokens];
    float* w = a.weights + bh * cap + j0 + tid;
#pragma unroll
    for (int i = 0; i < kWeightTokens; ++i) {
        sum[i] = 0.f;
        before[i] = j0 + tid + i * kFinishThreads < len ? w[i * kFinishThreads] : 0.f;
    }
    for (int rt = 0; rt < a.row_tiles; ++rt) {
        const int nrows = min(ROWS, a.rows - rt * ROWS);
        const float* sr = a.scores + scores_at<ROWS>(a, bh, rt, cap);
        const float* z = s_lse + rt * ROWS;
#pragma unroll
        for (int i = 0; i < kWeightTokens; ++i) {
            const int j = j0 + tid + i * kFinishThreads;
            if (j >= len) continue;
            const float* x = sr + (long long)j * nrows;
            if ((nrows & 3) == 0) {
                for (int r = 0; r < nrows; r += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(x + r);
                    sum[i] += (ex2(v.x - z[r]) + ex2(v.y - z[r + 1])) + (ex2(v.z - z[r + 2]) + ex2(v.w - z[r + 3]));
                }
            } else {
                for (int r = 0; r < nrows; ++r) sum[i] += ex2(x[r] - z[r]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kWeightTokens; ++i)
        if (j0 + tid + i * kFinishThreads < len) w[i * kFinishThreads] = before[i] + sum[i];
}

template <int D, int NB>
cudaError_t launch_d(const PagedDecodeFp8Launch& a, cudaStream_t s) {
    using C = Cfg<D, NB>;
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
    p.weights = a.weights;
    p.part_o = a.part_o;
    p.part_lse = a.part_lse;
    p.scores = a.weights ? a.scores : nullptr;
    p.prefix = a.prefix;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.Nq = a.Nq;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.rows = a.Hq / a.Hkv * a.Nq;
    p.row_tiles = (p.rows + C::ROWS - 1) / C::ROWS;
    p.blocks_per_page = (uint32_t)(a.page / a.sb);
    p.page = FastDiv((uint32_t)a.page);
    p.sb = FastDiv((uint32_t)a.sb);
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    const int cap = a.max_pages * a.page;
    const long long bh = (long long)a.B * a.Hkv;
    // no more CTAs than steps at full lengths
    p.workers = (int)std::min<long long>(a.workers, bh * p.row_tiles * ((cap + C::STEP - 1) / C::STEP));
    e = launch_dependent(decode_fp8_kernel<D, NB>, dim3(p.workers), dim3(kThreads), C::SMEM, s, p);
    if (e != cudaSuccess) return e;
    constexpr int per_block = kFinishThreads * kWeightTokens;
    const int weight_blocks = a.weights ? (cap + per_block - 1) / per_block : 0;
    const long long row_blocks = bh * p.rows, blocks = row_blocks + bh * weight_blocks;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    return launch_dependent(finish_fp8_kernel<D, C::ROWS>, dim3((unsigned)blocks), dim3(kFinishThreads),
                            a.weights ? (size_t)p.rows * 4 : 0, s, p, (unsigned)row_blocks, weight_blocks);
}

template <int D, int NB>
cudaError_t blocks_per_sm(int* blocks) {
    using C = Cfg<D, NB>;
    const cudaError_t e = set_smem_limit_once<decode_fp8_kernel<D, NB>>(C::SMEM);
    if (e != cudaSuccess) return e;
    const cudaError_t f = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, decode_fp8_kernel<D, NB>, kThreads, C::SMEM);
    *blocks = std::min(*blocks, C::CTAS);
    return f;
}

}  // namespace

cudaError_t launch_decode_paged_fp8(const PagedDecodeFp8Launch& a, cudaStream_t s) {
    const int tile = fp8_tile_rows(a.Hq / a.Hkv * a.Nq);
    if (a.d == 128) return tile == 8 ? launch_d<128, 1>(a, s) : tile == 16 ? launch_d<128, 2>(a, s) : launch_d<128, 4>(a, s);
    return tile == 8 ? launch_d<64, 1>(a, s) : tile == 16 ? launch_d<64, 2>(a, s) : launch_d<64, 4>(a, s);
}

cudaError_t decode_fp8_blocks_per_sm(int d, int tile, int* n) {
    if (d == 128) return tile == 8 ? blocks_per_sm<128, 1>(n) : tile == 16 ? blocks_per_sm<128, 2>(n) : blocks_per_sm<128, 4>(n);
    return tile == 8 ? blocks_per_sm<64, 1>(n) : tile == 16 ? blocks_per_sm<64, 2>(n) : blocks_per_sm<64, 4>(n);
}

}  // namespace fa
