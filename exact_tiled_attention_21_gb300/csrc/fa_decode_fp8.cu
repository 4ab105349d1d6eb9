// Attention of 1..16 new tokens per sequence over a paged cache held in 8 bits
// (e4m3 with one fp32 scale per block of sb tokens and kv head).
//
// Every byte of the cache is read once per 32 query rows (the Hq / Hkv heads of
// a group times the new tokens), 2 d bytes per key for 4 d flops per row: bound
// by HBM for 8 rows of d = 128 (5.2 TB/s, start and end included), by the latencies
// of widening and multiplying for more (32 rows: 2 warps per scheduler, 35% of the
// issue slots, a quarter of HBM's rate) and at d = 64.  A CTA has four
// warps.  Each streams 32 keys per step through a ring of cp.async copies and
// holds 8 query rows, or 16 where there are more, so that a widened fragment
// serves two products.  Up to 16 rows the warps take different keys and wait for
// nobody until the end; with 32 two warps read each other's keys, each for rows
// of its own.  8 sequences of 8000 tokens, 4 kv heads, d = 128, one token each, calls
// back to back: 20.7 us for 8 rows, 25.3 for 16, 33.7 for 32 (8 rows in each of four
// warps that share keys: 9% more, and 19% for 80 rows; 32 rows in every warp, the
// queries in shared memory: 20%).
//
// The work is one list of steps of 128 keys over all sequences, kv heads and row
// tiles, cut into equal shares for as many CTAs as run at once, from the lengths
// on the device: any batch of lengths, and any capacity of the block table, keeps
// every SM busy to the end.  A CTA's share crosses from one (sequence, kv head,
// row tile) to the next as it comes, the copies running ahead; the part of one
// that a CTA holds is a segment.  Segment results go to the workspace at slot
// CTA + item (which grows by one from each segment to the next) and a second
// kernel merges the segments of each row.
//
// The products are mma.sync m16n8k16 with fp16 operands and fp32 sums, because
// an e4m3 value is exact in fp16 and the fragments can be read straight from
// the cache's rows.  Both are taken transposed, S^T = K Q^T and O^T = V^T P^T,
// so that the keys (and d) fill the 16 rows of a product and the queries its 8
// columns.  The order of d within K Q^T and of the keys within V^T P^T is free: a
// lane's 16 consecutive bytes of a K row are the k-indices of its A fragments,
// and its d / 8 bytes of each of four V rows the k-pairs of its A fragments.  P
// turns from S^T's accumulators into the B fragments by an 8 x 8 transpose.
// tcgen05 would need the bytes widened and written back to shared memory first
// (the queries are not 8 bits wide), for 128-row products of at most 32 columns.
//
// q is scaled by a power of two per row into fp16's range (exact but for
// elements 2^-28 below the row's largest).  With x_j the score in log2 units,
// the softmax sums l = sum 2^(x_j - m) stay in fp32; the V product takes
// 2^(x_j + log2 vs_j - M) in fp16 with its own reference M, so that a block's
// scale can have any size.  M puts the largest weight between 2^11 and 2^15, as
// high as fp16 goes, so that the rounding is a relative 2^-11 (an eighth of the
// result's own bf16 step) down to 2^-25 of that weight and 2^-36 of it below: a
// long flat tail behind a token that takes almost all the weight keeps its value.
// (References at the maximum lost 12% of O for 65k tokens 2^23.6 below the first,
// where one warp has a quarter of them; 7 octaves below it with a slack of 8 took
// the same time.)  Result: O 2^(M - m) / l.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "fa_e4m3.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kKeys = 32, kStep = kWarps * kKeys;  // keys per warp and step, and per CTA
constexpr int kStages = 2;                         // steps in flight
constexpr float kSlack = 8.f;  // how far (log2) a score may exceed the reference that its softmax term is relative to
// The same for the value product, whose weights are fp16: the reference is set so that the largest one is 2^kTopV, and is
// kept until one would pass 2^(kTopV + kSlackV) = 2^15.  What lies below 2^-14 loses bits, so the range is put to use.
constexpr float kTopV = 11.f, kSlackV = 4.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

template <int D, int ROWS_>
struct Cfg {
    static constexpr int ROWS = ROWS_, NB = ROWS == 8 ? 1 : 2;  // query rows per tile; a warp's, in eights
    static constexpr int RG = ROWS / (8 * NB), KG = kWarps / RG;  // row groups; groups of warps with different keys
    static constexpr int HALF = kKeys * D;                 // bytes of K (and of V) per warp and step
    static constexpr int SLOT = 2 * HALF + 8 * kKeys;      // K, V, K scales, log2 of V scales
    static constexpr int RING = kStages * SLOT;            // per warp
    static constexpr int MERGE = kWarps * RING;            // byte offset of the merge buffers, one for each warp but the
                                                           // first group's
    static constexpr int OROW = D + 4;                     // a row of them, floats; within it column d (of 8 runs of
                                                           // D / 8: g, then 2 i + e) is at 16 i + 2 g + e: no bank conflicts
    static constexpr int SMEM = MERGE + (kWarps - RG) * 8 * NB * OROW * 4;
    // CTAs per SM, and those that the registers are made for; shared memory or registers must leave no room for one more,
    // or the next call's CTAs, started early, fill SMs unevenly (smaller merge buffers that let a third one in: 32 sequences
    // of 4096 tokens, calls back to back, 61.2 us against 52.4).  d = 128, up to 8 rows: bound by HBM, and a third CTA
    // only costs (128k tokens: 68 us with one, 55 with two, 58 with three; the copies alone 51 with one).  d = 64: bound
    // by instructions, four CTAs 28.9 us, three 30.2, five 30.6 (16 sequences of 3000 tokens, 16 heads).  16 rows per
    // warp take 249 registers at d = 128 and more than 128 at d = 64.
    static constexpr int CTAS = D == 64 ? 4 : 2, REGS_FOR = NB == 2 ? (D == 64 ? 3 : 2) : D == 64 ? 4 : 3;
    static_assert(CTAS * (SMEM + 1536) <= 227 * 1024, "shared memory");
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
    float* lse2;         // [B*Hq*Nq] log2 LSE of each row, with weights
    int B, Hq, Hkv, Nq, max_pages, num_pages, rows, row_tiles, workers;
    uint32_t blocks_per_page;
    FastDiv page, sb;
    float scale_log2;
    DevError* err;
};

__device__ __forceinline__ int clamp_len(int len, int cap) { return min(max(len, 0), cap); }

// Steps of all sequences before q (64-bit warp scan of the lengths): the sequence that step q falls in, its first step
// and length.  With q beyond the end: sequence B and the total.  prefix: also written, if not null.
__device__ __forceinline__ void find_sequence(const int* lens, int B, int cap, long long q, long long* prefix, int& b,
                                              long long& start, int& len) {
    const int lane = threadIdx.x & 31;
    long long base = 0;
    b = B;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int l = b0 + lane < B ? clamp_len(lens[b0 + lane], cap) : 0;
        const uint32_t n = (uint32_t)(l + kStep - 1) / kStep;
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

__device__ __forceinline__ void advance(Cursor& c, const Params& a, int cap) {
    if (++c.s < c.n) return;
    c.s = 0;
    if (++c.rt < a.row_tiles) return;
    c.rt = 0;
    if (++c.kvh < a.Hkv) return;
    c.kvh = 0;
    do {
        ++c.b;
        c.len = c.b < a.B ? clamp_len(a.lens[c.b], cap) : 0;
    } while (c.len == 0 && c.b < a.B);
    c.n = (c.len + kStep - 1) / kStep;
}

// Where the scores [key][rows of the tile] of a tile begin.  A (sequence, kv head)'s rows are padded to a multiple of
// four, so that a tile with a multiple of two or four rows has its scores of a key aligned to as many.
template <int ROWS>
__device__ __forceinline__ long long scores_at(const Params& a, long long bh, int rt, int cap) {
    return (bh * ((a.rows + 3) & ~3) + rt * ROWS) * cap;
}

// DRAFTS: more than one new token per sequence.  (8 sequences of 8000 tokens, 4 kv heads, d = 128, back to back: the code
// for keys that some rows do not see takes 26.3 us with 16 rows and 35.3 with 32, whether it runs or not; without it 25.3
// and 33.7.)
template <int D, int ROWS, bool DRAFTS>
__global__ void __launch_bounds__(kThreads, Cfg<D, ROWS>::REGS_FOR) decode_fp8_kernel(const Params a) {
    using C = Cfg<D, ROWS>;
    constexpr int MT = kKeys / 16, KS = D / 16, DT = D / 8, NB = C::NB, RG = C::RG, KG = C::KG;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_stat[kWarps][2][8 * NB];  // m and l of a warp's rows
    __shared__ Cursor s_ahead[kWarps];
    pdl_launch_dependents();
    pdl_wait();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rg = warp % RG, kg = warp / RG;  // row group, and group of warps that share keys
    const int P = (int)a.page.d, cap = a.max_pages * P, Nq = DRAFTS ? a.Nq : 1;
    if (blockIdx.x == 0)
        for (int i = tid; i < a.B; i += kThreads)
            if (a.lens[i] < 0 || a.lens[i] > cap) record_invalid(a.err, kSiteCacheLen, a.lens[i]);
    // ---- this CTA's share of the steps: `count` of them from `cur`
    const long long per_step = (long long)a.Hkv * a.row_tiles;
    Cursor cur;
    int count;
    {
        int b, len;
        long long total, start;
        find_sequence(a.lens, a.B, cap, LLONG_MAX, blockIdx.x == 0 && warp == 0 ? a.prefix : nullptr, b, total, len);
        total *= per_step;
        const long long workers = min((long long)a.workers, total);  // at least one step each
        if (blockIdx.x >= workers) return;
        const long long u = blockIdx.x * total / workers;
        count = (int)((blockIdx.x + 1ll) * total / workers - u);
        find_sequence(a.lens, a.B, cap, u / per_step, nullptr, cur.b, start, cur.len);
        cur.n = (cur.len + kStep - 1) / kStep;
        const long long in_b = u - start * per_step;
        const int item_b = (int)(in_b / cur.n);
        cur.s = (int)(in_b - (long long)item_b * cur.n);
        cur.kvh = item_b / a.row_tiles;
        cur.rt = item_b - cur.kvh * a.row_tiles;
    }

    // ---- Q fragments: k-step s of lane (g, t) is row g, columns (D = 128: 64 (s / 4) +) 16 t + 4 (s % 4) .. + 3
    uint32_t qb[NB][KS][2];
    float sc[NB][2];  // score scale of the rows whose scores this lane holds: 2 t, 2 t + 1 of each eight
    auto load_q = [&](int nb, uint32_t (&w)[D / 8]) {
        const int r = cur.rt * ROWS + (rg * NB + nb) * 8 + g;
        const uint4* src =
            reinterpret_cast<const uint4*>(a.q + (((long long)cur.b * a.Hkv + cur.kvh) * a.rows + r) * D + t * 16);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 x = r < a.rows ? src[i / 2 * 8 + i % 2] : make_uint4(0, 0, 0, 0);
            w[i * 4] = x.x, w[i * 4 + 1] = x.y, w[i * 4 + 2] = x.z, w[i * 4 + 3] = x.w;
        }
    };
    auto make_q = [&](int nb, const uint32_t (&w)[D / 8]) {
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // power of two that brings the row's largest element into [2^14, 2^15); rows of zeros, and of infinities (which
        // stay what they are), keep theirs
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
        for (int j = 0; j < 2; ++j) sc[nb][j] = __shfl_sync(0xffffffffu, up, (2 * t + j) * 4);
    };

    // ---- the ring: this warp's 32 keys of the steps ahead, whatever item they are of
    // A copy instruction moves whole rows (D / 16 lanes a row, so that a quarter warp asks for 128 consecutive bytes);
    // the fragments' readers find their 16 bytes (V at D = 64: 8) at
    //   K: (key / 8, half h of D = 128, lane' = 4 (key % 8) + t), lane' ^ 4 h
    //   V: (key / 16, r, 32-byte slot 4 s + (t ^ s), rest of the column), s = column / 32, at D = 64 t ^ s ^ 2 (r % 2),
    //   where key % 16 = 2 t + r % 2 + 8 (r / 2).
    // The exclusive-ors keep both the copies and the reads free of bank conflicts.  A 32-byte sector of a row stays
    // together: a copy whose sector is torn apart in shared memory fetches it from L2 once per piece (V in 16-byte
    // pieces: 1.5 times the bytes in all, which bound the kernel at 58 us of a 128k-token, 8-head cache).
    uint8_t* ring = smem + warp * C::RING;
    const uint32_t ring_u = smem_u32(ring);
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
    Cursor& ahead = s_ahead[warp];  // the step after `to_issue`; in shared memory to spare registers
    if (lane == 0) ahead = cur;
    __syncwarp();
    int fetched = 0, issued = 0;
    bool bad = false;
    struct {
        int page, key, len, kvh;  // the lane's key and its page, loaded one step before its use
    } to_issue;
    auto fetch_page = [&]() {
        to_issue.key = ahead.s * kStep + warp * kKeys + lane;
        to_issue.len = ahead.len;
        to_issue.kvh = ahead.kvh;
        to_issue.page = fetched < count && to_issue.key < ahead.len
                            ? a.table[(long long)ahead.b * a.max_pages + a.page.div(to_issue.key)]
                            : -1;
        if (++fetched < count) {
            Cursor next = ahead;
            advance(next, a, cap);
            __syncwarp();
            if (lane == 0) ahead = next;
            __syncwarp();
        }
    };
    // Scales are loaded, not copied (a 4-byte copy asks L2 once per lane, a load once per sector), and put into the
    // ring one step later, when they have arrived; V's as logarithms.  Plain loads here and of the lengths: the read-only
    // path is for data that stays as it is while the kernel runs, and this one starts before its wait for the append.
    float ks_next = 0.f, vs_next = 0.f;
    auto put_scales = [&](int slot, float ks, float vs) {
        float* f = reinterpret_cast<float*>(ring + slot * C::SLOT + 2 * C::HALF) + lane;
        f[0] = ks;
        f[kKeys] = lg2(vs);
    };
    // ALL: every key of the step is there.
    auto copy = [&](uint32_t base, uint32_t row, const bool ALL) {
#pragma unroll
        for (int n = 0; n < kKeys / RPI; ++n) {
            const uint32_t rr = __shfl_sync(0xffffffffu, row, n * RPI + cr);
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
    auto issue = [&](int slot, float& ks, float& vs) {
        if (issued < count) {
            const int key = to_issue.key, pg = to_issue.page;
            const bool in = key < to_issue.len, ok = in && (unsigned)pg < (unsigned)a.num_pages;
            bad |= in && !ok;
            const uint32_t at = (uint32_t)key - a.page.div(key) * P;
            const uint32_t head = (uint32_t)pg * a.Hkv + to_issue.kvh;
            const uint32_t row = ok ? head * P + at : ~0u;  // cache row of the lane's key, ~0 for none
            const uint32_t blk = ok ? head * a.blocks_per_page + a.sb.div(at) : 0u;
            ks = ok ? a.ks[blk] : 0.f;
            vs = ok ? a.vs[blk] : 0.f;
            if (__all_sync(0xffffffffu, ok))
                copy(ring_u + slot * C::SLOT, row, true);
            else
                copy(ring_u + slot * C::SLOT, row, false);
        }
        ++issued;
        cp_async_commit();
    };
    // a step's keys are read by the warps of the group
    auto group_sync = [&]() {
        if constexpr (RG == 1)
            __syncwarp();
        else if (RG == kWarps || kg == 0)
            bar_sync(1, RG * 32);
        else
            bar_sync(2, RG * 32);
    };
    // Where the D / 8 bytes of columns col D / 8 ... of a stage's key are, among the V bytes.
    auto v_piece = [&](int key, int col) {
        const int i = key / 16, t2 = key % 8 / 2, r = key % 2 + key % 16 / 8 * 2;
        if constexpr (D == 128) return ((i * 4 + r) * 16 + 4 * (col >> 1) + (t2 ^ (col >> 1))) * 32 + (col & 1) * 16;
        return ((i * 4 + r) * 8 + 4 * (col >> 2) + (t2 ^ ((col >> 2) | (r & 1) << 1))) * 32 + (col & 3) * 8;
    };
    // The high bits of the NaN bytes of a word of e4m3.
    auto nan_bytes = [](uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; };
    static_assert(kStages == 2, "the start");
    {   // the loads of the first steps depend on each other (lengths, pages, rows): the queries' come in between
        uint32_t w[NB][D / 8];
        fetch_page();
        const auto first = to_issue;
        fetch_page();
        const auto second = to_issue;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) load_q(nb, w[nb]);
        fetch_page();
        const auto third = to_issue;
        float ks = 0.f, vs = 0.f;
        to_issue = first;
        issue(0, ks, vs);
        to_issue = second;
        issue(1, ks_next, vs_next);
        to_issue = third;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) make_q(nb, w[nb]);
        put_scales(0, ks, vs);
    }

    // ---- the steps
    float acc[NB][D / 16][4];                // columns g d / 8 + 2 i + c / 2 of rows 2 t + c % 2 of each eight
    float m[NB][2], M[NB][2], l[NB][2];      // of rows 2 t + j; the references start at the lowest number: a row that sees
                                             // no key keeps l = 0 (2^(-inf - m))
    int seg = 0, slot = 0;                   // first step of the segment within its item; ring slot
    bool begins = true;
    for (int it = 0; it < count; ++it) {
        const int r0 = cur.rt * ROWS + rg * NB * 8, nrows = min(ROWS, a.rows - cur.rt * ROWS);  // of the warp, of the tile
        const long long bh = (long long)cur.b * a.Hkv + cur.kvh;
        if (begins) {
            seg = cur.s;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (it > 0) {
                    uint32_t w[D / 8];
                    load_q(nb, w);
                    make_q(nb, w);
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) acc[nb][i][0] = acc[nb][i][1] = acc[nb][i][2] = acc[nb][i][3] = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) m[nb][j] = M[nb][j] = -FLT_MAX, l[nb][j] = 0.f;
            }
        }
        cp_async_wait<kStages - 1>();
        group_sync();  // every lane's copies are there
        // A value product multiplies a key's V by the zero weights of the rows that do not see it, and 0 NaN is NaN.  Of
        // the keys that some rows do not see (the last Nq - 1) NaN bytes are put into the sums of the rows that do, and
        // become zeros in the stage.
        if (DRAFTS && cur.s * kStep + (kg + 1) * RG * kKeys > cur.len - Nq + 1) {
            const int part0 = kg * RG, base = cur.s * kStep + part0 * kKeys;  // the group's first key of this step
            const int from = max(cur.len - Nq + 1 - base, 0), to = min(cur.len - base, RG * kKeys);
            auto v_word = [&](int key, int col, int c) {  // columns col DT + 4 c .. + 3 of one of the group's keys
                return reinterpret_cast<uint32_t*>(smem + (part0 + key / kKeys) * C::RING + slot * C::SLOT + C::HALF +
                                                   v_piece(key % kKeys, col)) + c;
            };
            const int my = lane % (D / 4);  // the lane's word of a row
            bool nan = false;
            for (int key = from; key < to; ++key) nan |= nan_bytes(*v_word(key, my / (DT / 4), my % (DT / 4))) != 0;
            if (__any_sync(0xffffffffu, nan)) {  // in all warps of the group alike
#pragma unroll 1
                for (int key = from; key < to; ++key) {
                    const uint32_t* w = v_word(key, g, 0);
#pragma unroll
                    for (int c = 0; c < DT / 4; ++c) {
                        const uint32_t z = nan_bytes(w[c]);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const bool sees = base + key <= cur.len - Nq + (r0 + nb * 8 + 2 * t + j) % Nq;
#pragma unroll
                                for (int e = 0; e < 4; ++e)  // column 4 c + e
                                    if (sees && (z >> (8 * e + 7) & 1))
                                        acc[nb][2 * c + e / 2][e % 2 * 2 + j] = __int_as_float(0x7FFFFFFF);
                            }
                    }
                }
                group_sync();  // every warp has read them
#pragma unroll 1
                for (int key = from; key < to; ++key)
                    if (key / kKeys == rg && lane < D / 4) {
                        uint32_t* w = v_word(key, my / (DT / 4), my % (DT / 4));
                        *w &= ~((nan_bytes(*w) >> 7) * 0xFFu);
                    }
                group_sync();
            }
        }
#pragma unroll 1
        for (int part = 0; part < RG; ++part) {
            const int key0 = cur.s * kStep + (kg * RG + part) * kKeys;
            if (key0 >= cur.len || rg * NB * 8 >= nrows) break;
            const uint8_t* st = smem + (kg * RG + part) * C::RING + slot * C::SLOT;
            float S[NB][MT][4];  // keys 16 i + g, + 8 (c / 2) of rows 2 t + c % 2
            const uint4* kf = reinterpret_cast<const uint4*>(st);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < MT; ++i) S[nb][i][0] = S[nb][i][1] = S[nb][i][2] = S[nb][i][3] = 0.f;
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
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const uint32_t ka[4] = {e4m3x2_to_half2(w[2 * i][c]), e4m3x2_to_half2(w[2 * i + 1][c]),
                                                e4m3x2_hi_to_half2(w[2 * i][c]), e4m3x2_hi_to_half2(w[2 * i + 1][c])};
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_16816(S[nb][i], ka, qb[nb][h * 4 + c][0], qb[nb][h * 4 + c][1]);
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
                        S[nb][i][2 * h] *= sc[nb][0] * kscale;
                        S[nb][i][2 * h + 1] *= sc[nb][1] * kscale;
                    }
                }
            uint32_t pb[NB][MT][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                auto& x = S[nb];
                if (key0 + kKeys > cur.len - Nq + 1) {  // some row does not see every key
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int lim = cur.len - Nq + (r0 + nb * 8 + 2 * t + j) % Nq + 1 - key0 - g;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (i * 16 + h * 8 >= lim) x[i][2 * h + j] = -INFINITY;
                    }
                }
                if (a.scores) {  // [key][row of the tile]: a lane's two rows are neighbours
                    const int r = (rg * NB + nb) * 8 + 2 * t;
                    float* sr = a.scores + scores_at<ROWS>(a, bh, cur.rt, cap) + (long long)(key0 + g) * nrows + r;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (key0 + i * 16 + h * 8 + g < cur.len) {
                                float* at = sr + (i * 16 + h * 8) * nrows;
                                if ((nrows & 1) == 0) {
                                    if (r < nrows) *reinterpret_cast<float2*>(at) = make_float2(x[i][2 * h], x[i][2 * h + 1]);
                                } else {
                                    if (r < nrows) at[0] = x[i][2 * h];
                                    if (r + 1 < nrows) at[1] = x[i][2 * h + 1];
                                }
                            }
                }
                // ---- softmax: p = 2^(x - m) into l; w = 2^(x + log2 vs - M) for the value product.  m need not be the
                // maximum, only within 2^8 of it, and M not 2^11 below, only within 2^4 of that: most steps find no larger
                // one and skip the reductions.
                float mx[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[j] = fmaxf(x[0][j], x[0][2 + j]);
#pragma unroll
                    for (int i = 1; i < MT; ++i) mx[j] = fmax3(mx[j], x[i][j], x[i][2 + j]);
                }
                if (__any_sync(0xffffffffu, mx[0] > m[nb][0] + kSlack || mx[1] > m[nb][1] + kSlack)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = fmaxf(m[nb][j], mx[j]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        l[nb][j] *= ex2(m[nb][j] - top);
                        m[nb][j] = top;
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float lv = ksf[kKeys + i * 16 + h * 8];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            l[nb][j] += ex2(x[i][2 * h + j] - m[nb][j]);
                            x[i][2 * h + j] += lv;
                        }
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[j] = fmaxf(x[0][j], x[0][2 + j]);
#pragma unroll
                    for (int i = 1; i < MT; ++i) mx[j] = fmax3(mx[j], x[i][j], x[i][2 + j]);
                }
                if (__any_sync(0xffffffffu, mx[0] > M[nb][0] + (kTopV + kSlackV) || mx[1] > M[nb][1] + (kTopV + kSlackV))) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = fmaxf(M[nb][j], mx[j] - kTopV);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const float f = ex2(M[nb][j] - top);
                        M[nb][j] = top;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            acc[nb][i][j] *= f;
                            acc[nb][i][2 + j] *= f;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const __half2 w = __floats2half2_rn(ex2(x[i][2 * h] - M[nb][0]), ex2(x[i][2 * h + 1] - M[nb][1]));
                        pb[nb][i][h] = transpose8x8(*reinterpret_cast<const uint32_t*>(&w));
                    }
            }
            const uint8_t* vf = st + C::HALF;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t v[4][DT / 4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4*>(
                            vf + ((i * 4 + r) * 16 + 4 * (g >> 1) + (t ^ (g >> 1))) * 32 + (g & 1) * 16);
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
                        for (int nb = 0; nb < NB; ++nb) mma_16816(acc[nb][2 * c + h], va, pb[nb][i][0], pb[nb][i][1]);
                    }
            }
        }
        put_scales(slot ^ 1, ks_next, vs_next);
        group_sync();  // every lane has read this slot
        issue(slot, ks_next, vs_next);
        fetch_page();
        slot ^= 1;

        // ---- at the segment's end: O = sum over the warps with these rows of O_w 2^(M_w - m) / l.  The factor meets
        // O_w as two, 2^((M_w - m) / 2) and the same / l: O is in range where O l is not (values near the largest bf16
        // number), or where 2^(M_w - m) is not (below 2^-126 or subnormal, where every block has the smallest scale).
        const bool item_ends = cur.s + 1 == cur.n;
        begins = item_ends || it + 1 == count;
        if (begins) {
            float f[NB][2], fl[NB][2];
            auto factors = [](float M, float m, float l, float& f, float& fl) {
                f = ex2(0.5f * (M - m));
                fl = l == 0.f ? 0.f : f / l;  // 0: the row sees no key; NaN stays
            };
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], d);
                    const int r = nb * 8 + 2 * t + j;
                    if (KG > 1 && g == 0) s_stat[warp][0][r] = m[nb][j], s_stat[warp][1][r] = l[nb][j];
                    if (KG == 1) factors(M[nb][j], m[nb][j], l[nb][j], f[nb][j], fl[nb][j]);
                }
            if constexpr (KG > 1) {
                __syncthreads();
                float* buf = reinterpret_cast<float*>(smem + C::MERGE) + g * 2;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = nb * 8 + 2 * t + j;
                        float top = m[nb][j], sum = 0.f;
#pragma unroll
                        for (int w = 0; w < KG; ++w) top = fmaxf(top, s_stat[w * RG + rg][0][r]);
#pragma unroll
                        for (int w = 0; w < KG; ++w)
                            sum += s_stat[w * RG + rg][1][r] * ex2(s_stat[w * RG + rg][0][r] - top);
                        factors(M[nb][j], top, sum, f[nb][j], fl[nb][j]);
                        m[nb][j] = top;
                        l[nb][j] = sum;
                        if (kg > 0)
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
                                *reinterpret_cast<float2*>(buf + ((warp - RG) * 8 * NB + r) * C::OROW + i * 16) =
                                    make_float2(acc[nb][i][j] * f[nb][j] * fl[nb][j],
                                                acc[nb][i][2 + j] * f[nb][j] * fl[nb][j]);
                    }
                __syncthreads();
                if (kg == 0) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                float2 x = make_float2(acc[nb][i][j] * f[nb][j] * fl[nb][j],
                                                       acc[nb][i][2 + j] * f[nb][j] * fl[nb][j]);
#pragma unroll
                                for (int w = 1; w < KG; ++w) {
                                    const float2 y = *reinterpret_cast<const float2*>(
                                        buf + (((w - 1) * RG + rg) * 8 * NB + nb * 8 + 2 * t + j) * C::OROW + i * 16);
                                    x.x += y.x;
                                    x.y += y.y;
                                }
                                acc[nb][i][j] = x.x;
                                acc[nb][i][2 + j] = x.y;
                            }
                            f[nb][j] = fl[nb][j] = 1.f;
                        }
                }
            }
            if (kg == 0) {
                const bool whole = seg == 0 && item_ends;
                const long long slot_out = blockIdx.x + bh * a.row_tiles + cur.rt;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = (rg * NB + nb) * 8 + 2 * t + j;
                        if (r >= nrows) continue;
                        const float sum = l[nb][j];
                        const float lse2 = sum == 0.f ? -INFINITY : m[nb][j] + lg2(sum);
                        const long long row = bh * a.rows + cur.rt * ROWS + r;  // (b, head, token) flattened
                        float o[DT];
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            o[2 * i] = acc[nb][i][j] * f[nb][j] * fl[nb][j],
                                  o[2 * i + 1] = acc[nb][i][2 + j] * f[nb][j] * fl[nb][j];
                        if (whole) {
                            uint4* dst = reinterpret_cast<uint4*>(a.o + row * D + g * DT);
#pragma unroll
                            for (int i = 0; i < DT / 8; ++i)
                                dst[i] = make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                                                    pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
                            if (a.lse && g == 0) a.lse[row] = lse2 * kLn2;
                            if (a.weights && g == 0) a.lse2[row] = lse2;
                        } else {
                            float4* dst = reinterpret_cast<float4*>(a.part_o + (slot_out * ROWS + r) * D + g * DT);
#pragma unroll
                            for (int i = 0; i < DT / 4; ++i)
                                dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            if (g == 0) a.part_lse[slot_out * ROWS + r] = lse2;
                        }
                    }
            }
        }
        if (it + 1 < count) advance(cur, a, cap);
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
#pragma unroll 4
    for (int s = lane; s < segs; s += 32) M = fmaxf(M, pl[(long long)s * stride]);
    for (int w = 16; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    base = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
#pragma unroll 4
    for (int s = lane; s < segs; s += 32) sum += ex2(pl[(long long)s * stride] - base);
    for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    return sum;
}

// One block per run of `run` rows of a tile, one after the other: LSE = M + log2 sum 2^(lse_s - M), O = sum 2^(lse_s - M)
// o_s / sum, the segments dealt to groups of D / 4 threads.  A row without keys gets O = 0, LSE = -inf; rows whose item was
// one segment are already written.  Of rows in longer runs with few segments a group takes one each (47 sequences of 1200
// tokens, 2 heads, 80 rows: 7.7 us, one after the other 13.4); single rows are faster with the groups sharing the segments
// (one sequence of 777 tokens: 10.3 us in all against 12.3).  Bound by latency.
template <int D, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) finish_fp8_kernel(const Params a, int run, int runs) {
    constexpr int LANES = D / 4, GROUPS = THREADS / LANES, AHEAD = 4;
    __shared__ float4 s_o[GROUPS][LANES];
    pdl_wait();
    // The last kernel of a call starts nothing early: the next call's CTAs, sharing SMs with this one's, would begin
    // unevenly (32 sequences of 4096 tokens, 8 heads, d = 64, calls back to back: 39.4 us against 31.6).
    if (a.weights) pdl_launch_dependents();
    const int tid = threadIdx.x, grp = tid / LANES, col = tid % LANES;
    const long long bh = blockIdx.x / runs;
    const int r0 = (int)(blockIdx.x % runs) * run, b = (int)(bh / a.Hkv), rt = r0 / ROWS;
    long long slot = 0;
    const int segs = find_segments(a, b, (int)(bh % a.Hkv) * a.row_tiles + rt, slot);
    auto write = [&](long long row, float4 o, float sum, float base) {
        *reinterpret_cast<uint2*>(a.o + row * D + col * 4) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
        if (col > 0) return;
        const float lse2 = sum == 0.f ? -INFINITY : base + lg2(sum);
        if (a.lse) a.lse[row] = lse2 * kLn2;
        if (a.weights) a.lse2[row] = lse2;
    };
    if (segs == 1) return;
    if (run > 1 && segs <= AHEAD) {  // a group for each row
        for (int r = r0 + grp; r < min(r0 + run, a.rows); r += GROUPS) {
            const long long at = slot * ROWS + (r - rt * ROWS), row = bh * a.rows + r;
            float4 v[AHEAD];
            float w[AHEAD], top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) {
                w[s] = s < segs ? a.part_lse[at + s * ROWS] : -INFINITY;
                v[s] = s < segs ? reinterpret_cast<const float4*>(a.part_o + (at + s * ROWS) * D)[col]
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) top = fmaxf(top, w[s]);
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) sum += w[s] = ex2(w[s] - base);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) {
                o.x = fmaf(w[s] * inv, v[s].x, o.x);
                o.y = fmaf(w[s] * inv, v[s].y, o.y);
                o.z = fmaf(w[s] * inv, v[s].z, o.z);
                o.w = fmaf(w[s] * inv, v[s].w, o.w);
            }
            write(row, o, sum, base);
        }
        return;
    }
    for (int r = r0; r < min(r0 + run, a.rows); ++r) {
        const long long at = slot * ROWS + (r - rt * ROWS), row = bh * a.rows + r;
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
        if (r > r0) __syncthreads();  // the row before is read
        s_o[grp][col] = o;
        __syncthreads();
        if (grp > 0) continue;
#pragma unroll
        for (int i = 1; i < GROUPS; ++i) {
            const float4 x = s_o[i][col];
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
        }
        write(row, o, sum, base);
    }
}

// weights[j] += sum over the rows of 2^(x_j - LSE), in a fixed order.  A block takes up to 1024 tokens, row tile after row
// tile.  With 4, 8, 16 or 32 rows in a tile a token's scores are 16-byte pieces of 1, 2, 4 or 8 lanes; else a thread reads
// its token's.  (That for all: 7 sequences of 30000 tokens, 2 kv heads, 80 rows 119 us against 31, 4.4 TB/s; with 4 rows,
// 32 sequences of 4096 tokens, 8 kv heads, the whole decode 71.6 us against 70.4.)
constexpr int kWeightThreads = 256, kPart = 4096, kPieces = kPart / 4 / kWeightThreads;  // scores of a block and tile

template <int ROWS>
__global__ void __launch_bounds__(kWeightThreads) weights_fp8_kernel(const Params a, int blocks, int tokens) {
    __shared__ float s_sum[kPart / 4];
    pdl_wait();
    const int tid = threadIdx.x, cap = a.max_pages * (int)a.page.d;
    const long long bh = blockIdx.x / blocks;
    const int len = clamp_len(a.lens[bh / a.Hkv], cap), begin = (int)(blockIdx.x % blocks) * tokens;
    const int many = min(tokens, len - begin);
    if (many <= 0) return;
    float* weights = a.weights + bh * cap + begin;
    float before[kPieces];
#pragma unroll
    for (int q = 0; q < kPieces; ++q)
        if (tid + q * kWeightThreads < many) before[q] = weights[tid + q * kWeightThreads];
    for (int rt = 0; rt < a.row_tiles; ++rt) {
        const int nrows = min(ROWS, a.rows - rt * ROWS);
        const float* scores = a.scores + scores_at<ROWS>(a, bh, rt, cap) + (long long)begin * nrows;
        const float* lse2 = a.lse2 + bh * a.rows + rt * ROWS;
        const bool vec = nrows >= 4 && (nrows & (nrows - 1)) == 0;
        const int lanes = vec ? nrows / 4 : 1, shift = __ffs(lanes) - 1, lane = tid & (lanes - 1);
        float sum[kPieces] = {};
        if (vec) {
            float4 x[kPieces];
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
                if ((tid + q * kWeightThreads) >> shift < many)
                    x[q] = reinterpret_cast<const float4*>(scores)[tid + q * kWeightThreads];
            float z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float l = lse2[lane * 4 + i];
                z[i] = l == -INFINITY ? INFINITY : l;  // a row without keys: every weight 2^-inf = 0
            }
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
                sum[q] = (ex2(x[q].x - z[0]) + ex2(x[q].y - z[1])) + (ex2(x[q].z - z[2]) + ex2(x[q].w - z[3]));
                for (int w = lanes / 2; w >= 1; w >>= 1) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], w);
            }
        } else {
            for (int r = 0; r < nrows; ++r) {
                const float l = lse2[r], z = l == -INFINITY ? INFINITY : l;
#pragma unroll
                for (int q = 0; q < kPieces; ++q) {
                    const int j = tid + q * kWeightThreads;
                    if (j < many) sum[q] += ex2(scores[j * nrows + r] - z);
                }
            }
        }
        if (rt > 0) __syncthreads();
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int j = (tid + q * kWeightThreads) >> shift;
            if (lane == 0 && j < many) s_sum[j] = rt > 0 ? s_sum[j] + sum[q] : sum[q];
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
        const int j = tid + q * kWeightThreads;
        if (j < many) weights[j] = before[q] + s_sum[j];
    }
}

template <int D, int ROWS>
cudaError_t launch_d(const PagedDecodeFp8Launch& a, cudaStream_t s) {
    using C = Cfg<D, ROWS>;
    cudaError_t e = a.Nq > 1 ? set_smem_limit_once<decode_fp8_kernel<D, ROWS, true>>(C::SMEM)
                             : set_smem_limit_once<decode_fp8_kernel<D, ROWS, false>>(C::SMEM);
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
    p.lse2 = a.lse2;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.Nq = a.Nq;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.rows = a.Hq / a.Hkv * a.Nq;
    p.row_tiles = (p.rows + ROWS - 1) / ROWS;
    p.blocks_per_page = (uint32_t)(a.page / a.sb);
    p.page = FastDiv((uint32_t)a.page);
    p.sb = FastDiv((uint32_t)a.sb);
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    const int cap = a.max_pages * a.page;
    const long long bh = (long long)a.B * a.Hkv;
    // no more CTAs than steps at full lengths
    p.workers = (int)std::min<long long>(a.workers, bh * p.row_tiles * ((cap + kStep - 1) / kStep));
    e = launch_dependent(a.Nq > 1 ? decode_fp8_kernel<D, ROWS, true> : decode_fp8_kernel<D, ROWS, false>, dim3(p.workers),
                         dim3(kThreads), C::SMEM, s, p);
    if (e != cudaSuccess) return e;
    // rows per finishing block: one up to 16 blocks per SM (45 sequences of 20 tokens, 8 heads, 80 rows: 32.5 us with one,
    // 5.0 with 16); its threads: 512 where an item has 32 segments or more (a single one of 70000 tokens, 16 rows: 17.7 us
    // with 128, 11.2 with 512; 8 of 128k tokens the same)
    int run = 1;
    while (run < ROWS && bh * p.rows > 16ll * run * a.num_sms) run *= 2;
    const int runs = (p.rows + run - 1) / run;
    const dim3 rows((unsigned)(bh * runs));
    e = p.workers >= 32 * bh * p.row_tiles
            ? launch_dependent(finish_fp8_kernel<D, ROWS, 512>, rows, dim3(512), 0, s, p, run, runs)
            : launch_dependent(finish_fp8_kernel<D, ROWS, 128>, rows, dim3(128), 0, s, p, run, runs);
    if (e != cudaSuccess || !a.weights) return e;
    int tokens = kPart / 4;  // of a block: as many as its rows leave room for
    while (tokens * std::min(p.rows, ROWS) > kPart) tokens /= 2;
    const int blocks = (cap + tokens - 1) / tokens;
    return launch_dependent(weights_fp8_kernel<ROWS>, dim3((unsigned)(bh * blocks)), dim3(kWeightThreads), 0, s, p, blocks,
                            tokens);
}

template <int D, int ROWS, bool DRAFTS>
cudaError_t resident(int* blocks) {
    using C = Cfg<D, ROWS>;
    const cudaError_t e = set_smem_limit_once<decode_fp8_kernel<D, ROWS, DRAFTS>>(C::SMEM);
    if (e != cudaSuccess) return e;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, decode_fp8_kernel<D, ROWS, DRAFTS>, kThreads, C::SMEM);
}

template <int D, int ROWS>
cudaError_t blocks_per_sm(int* blocks) {
    int one = 0, drafts = 0;
    cudaError_t e = resident<D, ROWS, false>(&one);
    if (e == cudaSuccess) e = resident<D, ROWS, true>(&drafts);
    *blocks = std::min({one, drafts, Cfg<D, ROWS>::CTAS});
    return e;
}

}  // namespace

cudaError_t launch_decode_paged_fp8(const PagedDecodeFp8Launch& a, cudaStream_t s) {
    const int tile = fp8_tile_rows(a.Hq / a.Hkv * a.Nq);
    if (a.d == 128) return tile == 8 ? launch_d<128, 8>(a, s) : tile == 16 ? launch_d<128, 16>(a, s) : launch_d<128, 32>(a, s);
    return tile == 8 ? launch_d<64, 8>(a, s) : tile == 16 ? launch_d<64, 16>(a, s) : launch_d<64, 32>(a, s);
}

cudaError_t decode_fp8_blocks_per_sm(int d, int tile, int* n) {
    if (d == 128) return tile == 8 ? blocks_per_sm<128, 8>(n) : tile == 16 ? blocks_per_sm<128, 16>(n) : blocks_per_sm<128, 32>(n);
    return tile == 8 ? blocks_per_sm<64, 8>(n) : tile == 16 ? blocks_per_sm<64, 16>(n) : blocks_per_sm<64, 32>(n);
}

}  // namespace fa
