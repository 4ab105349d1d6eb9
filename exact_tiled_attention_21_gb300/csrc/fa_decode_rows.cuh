// Attention of 1..16 new tokens per sequence over the paged bf16 cache: over the
// blocks of a list, or over the tokens that follow a prefix which all sequences
// share.  The prefix itself is fa_prefix.cu's, which with few rows of a sequence and kv
// head runs this beside it; or, where all sequences together have few query rows per
// kv head and little to share, it is one more sequence here for each 32 of them.
//
// 4 d bytes per key for 4 d flops per query row: bound by HBM.  The work is one
// list of steps of 4 x KEYS keys over all sequences, kv heads and row tiles, cut
// into equal shares for as many CTAs as run at once, from the lengths on the
// device: a batch of any lengths keeps every SM busy to the end.  A CTA's share
// crosses from one (sequence, kv head, row tile) to the next as it comes, the
// copies running ahead; the part of one that a CTA holds is a segment.  Segment
// results go to the workspace at slot CTA + item (which grows by one from each
// segment to the next), and a second kernel (fa_decode_rows.cu) merges the segments of
// each row.
//
// Where a list's items are few enough for a CTA of their own each, a cluster of up to
// eight takes an item, a run of its steps each, and joins the parts through its
// shared memories: no second kernel.
//
// Measured: 64 listed blocks of 16 tokens for each of 32 sequences, 4 heads on each of 8
// kv heads, d = 128: 25.4 us, 19.3 at HBM's copy rate; 128 blocks 49 us under the
// profiler, at about 70% of DRAM's peak.  What is left is the start (three loads that depend on
// one another behind the launch), the unequal ends and the join.
//
// A CTA has four warps.  Each streams KEYS keys per step through a ring of its own
// of cp.async copies, three steps deep, and holds 8 query rows, or 16 where there
// are more; with 32 two warps read each other's keys, each for rows of its own.
// Up to 16 rows the warps wait for nobody until a segment's end.
//
// The products are mma.sync m16n8k16 in bf16 with fp32 sums, taken transposed,
// S^T = K Q^T and O^T = V^T P^T, so that keys (and d) fill the 16 rows of a product
// and the queries its 8 columns: with a handful of query rows per kv head the
// 128-row products of tcgen05 would be nearly empty, and its operands would have to
// pass through shared memory again.  Softmax sums are fp32.  A row's weights are
// taken relative to a running reference within 2^8 of its largest score, and enter
// the value product as bf16 pairs of a rounded weight and what the rounding left:
// one bf16 (2^-8) would cost as much as the rounding of the result; of a pair the
// second number, below 2^-8 of the weight, is off by half a step, 2^-17 of it.
#pragma once
#include <algorithm>
#include <cfloat>
#include <climits>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kStages = 3;
constexpr float kSlack = 8.f;  // how far (log2) a score may exceed the reference that its weight is relative to
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// 16 bytes into shared memory; zeros if !ok (src must still be a valid address).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

template <int D, int ROWS_>
struct Cfg {
    static constexpr int ROWS = ROWS_, NB = ROWS == 8 ? 1 : 2;   // query rows per tile; a warp's, in eights
    static constexpr int RG = ROWS / (8 * NB), KG = kWarps / RG;  // row groups; groups of warps with different keys
    static constexpr int KEYS = D == 128 ? 16 : 32;              // per warp and step
    static constexpr int STEP = kWarps * KEYS;                   // per CTA
    static constexpr int HALF = KEYS * D * 2;                    // bytes of K (and of V) per warp and step
    static constexpr int SLOT = 2 * HALF + 128;                  // K, V, the keys' tokens
    static constexpr int RING = kStages * SLOT;                  // per warp
    static constexpr int OROW = D + 4;                           // a row of the merge buffers, floats
    static constexpr int MERGE = kWarps * RING;                  // one of 8 rows for each warp but the first group's
    static constexpr int SMEM = MERGE + (kWarps - RG) * 8 * OROW * 4;
    static constexpr int CTAS = 2;                               // per SM
    static_assert(CTAS * (SMEM + 2048) <= 227 * 1024, "shared memory");
    static_assert(HALF == 4096, "the swizzle's offsets");
};

struct Params {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kp;
    const __nv_bfloat16* vp;
    const int* table;
    const int* lens;
    const int* list;        // [B, Hkv, keep] blocks, or null: the tokens behind the shared ones
    const int* shared;      // [1], null with a list
    __nv_bfloat16* o;
    float* lse;
    float* part_o;          // [slot][ROWS][D], normalised
    float* part_lse;        // [slot][ROWS], log2
    int* ends;              // [item][2]: the CTAs of its first and last step
    const float* pre_o;     // the shared prefix's parts: [slot][pre_rows][D] and [slot][pre_rows], and ends as above
    const float* pre_lse;
    const int* pre_ends;
    int B, Hkv, Nq, max_pages, num_pages, rows, row_tiles, workers, keep;
    int cluster;            // CTAs of an item (LIST), 0: shares of all items' steps
    int pre_workers, pre_tiles, pre_rows, pre_item;  // its CTAs; its tiles of pre_rows query rows; the first one's slots are
                                                     // CTA + pre_item
    int joint, tiles;       // the prefix is this kernel's too: `joint` rows, as `tiles` sequences B, B + 1, ... of ROWS each
    FastDiv page, block, per_row, heads;  // rows, Hkv
    float scale_log2;
    DevError* err;
};

__host__ __device__ __forceinline__ int clamp_len(int len, int cap) { return min(max(len, 0), cap); }

// The shared tokens that sequences of these lengths read from the common prefix: none if some new token of it does not see
// all of them.
__host__ __device__ __forceinline__ int shared_of(int shared, int len, int Nq) { return len - Nq >= shared ? shared : 0; }

// A sequence's keys in this pass.
template <bool LIST>
__host__ __device__ __forceinline__ int keys_of(const Params& a, int len, int shared) {
    if constexpr (LIST) {
        return min(a.keep, (int)a.block.div(len + a.block.d - 1)) * (int)a.block.d;
    } else {
        return len - shared_of(shared, len, a.Nq);
    }
}

// The same of any place in the list of sequences; from B on it is the prefix, if that is this kernel's: every row sees all
// of it.
template <bool LIST>
__device__ __forceinline__ int length_of(const Params& a, int b, int cap, int shared) {
    if (b < a.B) return clamp_len(a.lens[b], cap);
    return !LIST && b < a.B + a.tiles ? shared + a.Nq : 0;
}
template <bool LIST>
__device__ __forceinline__ int keys_in(const Params& a, int b, int len, int shared) {
    if (!LIST && b >= a.B) return b < a.B + a.tiles ? shared : 0;
    return keys_of<LIST>(a, len, shared);
}

// What an item costs besides its steps, in steps: its queries, and joining its parts (64 sequences of 2 to 1000 own tokens, 8
// kv heads: the CTAs that got the shortest ones took 53 us, the others 25).
constexpr uint32_t kItemCost = 1;

// A warp's worth of sequences from b0 on: a lane's length, steps (of each of its items) and the sums up to it, of costs and
// of steps.
struct Scan {
    int len;
    uint32_t n, cost, steps;
};
template <int STEP, bool LIST>
__device__ __forceinline__ Scan scan_at(const Params& a, int cap, int shared, int b0) {
    const int lane = threadIdx.x & 31;
    Scan x;
    x.len = length_of<LIST>(a, b0 + lane, cap, shared);
    x.n = (uint32_t)(keys_in<LIST>(a, b0 + lane, x.len, shared) + STEP - 1) / STEP;
    x.steps = x.n;
    x.cost = x.n ? x.n + kItemCost : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t s = __shfl_up_sync(0xffffffffu, x.steps, d), c = __shfl_up_sync(0xffffffffu, x.cost, d);
        if (lane >= d) x.steps += s, x.cost += c;
    }
    return x;
}

// The steps and costs of all sequences, of one item each.
template <int STEP, bool LIST>
__device__ __forceinline__ uint2 cost_of_all(const Params& a, int cap, int shared) {
    uint2 total = make_uint2(0, 0);
    for (int b0 = 0; b0 < a.B + (LIST ? 0 : a.tiles); b0 += 32) {
        const Scan x = scan_at<STEP, LIST>(a, cap, shared, b0);
        total.x += __shfl_sync(0xffffffffu, x.steps, 31);
        total.y += __shfl_sync(0xffffffffu, x.cost, 31);
    }
    return total;
}

// A position in the list of steps.
struct Cursor {
    int b, len, keys, n;  // sequence (from B on the prefix), its length, its keys in this pass and their steps
    int kvh, rt, s;       // kv head, row tile and step
};

template <int STEP, bool LIST>
__device__ __forceinline__ void advance(Cursor& c, const Params& a, int cap, int shared) {
    if (++c.s < c.n) return;
    c.s = 0;
    if (++c.rt < a.row_tiles) return;
    c.rt = 0;
    if (++c.kvh < a.Hkv) return;
    c.kvh = 0;
    do {
        ++c.b;
        c.len = length_of<LIST>(a, c.b, cap, shared);
        c.keys = keys_in<LIST>(a, c.b, c.len, shared);
    } while (c.keys == 0 && c.b < a.B + (LIST ? 0 : a.tiles));
    c.n = (c.keys + STEP - 1) / STEP;
}

constexpr int kMostCluster = 8;
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(mapa_shared(addr, rank))
                 : "memory");
    return v;
}

constexpr int kNone = INT_MAX;  // in the place of a token: no such key

template <int ROWS>
struct RowsShared {
    float stat[kWarps][2][ROWS == 8 ? 8 : 16];  // m and l of a warp's rows
    Cursor ahead[kWarps];
};

// Lengths out of range, noted by one CTA.
__device__ __forceinline__ void check_lengths(const int* lens, int B, int cap, int given, DevError* err) {
    for (int i = threadIdx.x; i < B; i += blockDim.x)
        if (lens[i] < 0 || lens[i] > cap) record_invalid(err, kSiteCacheLen, lens[i]);
    if ((given < 0 || given > cap) && threadIdx.x == 0) record_invalid(err, kSiteCacheLen, given);
}

// What CTA `cta` of `workers` does, by four warps; kThreads threads, of which this is number `tid`.  DRAFTS: more than one new
// token per sequence.  PART: these are four of the CTA's warps, which meet at barrier `bar`.
template <int D, int ROWS, bool DRAFTS, bool LIST, bool PART>
__device__ __forceinline__ void decode_rows(const Params& a, uint8_t* smem, RowsShared<ROWS>& sh, const int tid, const int cta,
                                            const int workers, const int bar) {
    using C = Cfg<D, ROWS>;
    constexpr int KEYS = C::KEYS, MT = KEYS / 16, KS = D / 16, NB = C::NB, RG = C::RG, KG = C::KG, STEP = C::STEP;
    static_assert(!PART || RG == 1, "barriers 1 and 2 are a row group's");
    auto sync = [&]() {
        if constexpr (PART)
            bar_sync(bar, kThreads);
        else
            __syncthreads();
    };
    const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rg = warp % RG, kg = warp / RG;  // row group, and group of warps that share keys
    const int P = (int)a.page.d, cap = a.max_pages * P, Nq = DRAFTS ? a.Nq : 1;
    const int given = LIST ? 0 : *a.shared;
    int shared = clamp_len(given, cap);
    int from = 0;  // the prefix is read through this sequence's row of the table, the first one that sees all of it
    if (!LIST && a.joint) {
        uint32_t hit = 0;
        for (int b0 = 0; b0 < a.B && !hit; b0 += 32) {
            hit = __ballot_sync(0xffffffffu, b0 + lane < a.B && clamp_len(a.lens[min(b0 + lane, a.B - 1)], cap) - Nq >= shared);
            from = b0 + __ffs(hit) - 1;
        }
        if (!hit) shared = 0;  // nobody does
    }
    // ---- this CTA's share of the steps: `count` of them from `cur`
    const uint32_t per_step = (uint32_t)a.Hkv * a.row_tiles;
    Cursor cur;
    int count;
    if (LIST && a.cluster) {  // a part of one item, perhaps none
        const uint32_t item = blockIdx.x / (uint32_t)a.cluster, bh = item / (uint32_t)a.row_tiles;
        cur.b = (int)a.heads.div(bh);
        cur.kvh = (int)bh - cur.b * a.Hkv;
        cur.rt = (int)(item - bh * a.row_tiles);
        cur.len = clamp_len(a.lens[cur.b], cap);
        cur.keys = keys_of<LIST>(a, cur.len, shared);
        cur.n = (cur.keys + STEP - 1) / STEP;
        const Share mine = share_of((uint32_t)cur.n, a.cluster, blockIdx.x % (uint32_t)a.cluster);
        cur.s = (int)mine.first;
        count = (int)mine.count;
    } else {
        const Scan head = scan_at<STEP, LIST>(a, cap, shared, 0);
        uint32_t total = __shfl_sync(0xffffffffu, head.cost, 31);
        const int all = a.B + (LIST ? 0 : a.tiles);
        for (int b0 = 32; b0 < all; b0 += 32) total += __shfl_sync(0xffffffffu, scan_at<STEP, LIST>(a, cap, shared, b0).cost, 31);
        const Share mine = share_of(total * per_step, workers, cta);
        // the steps before a place in the list of costs, and the item and step there
        auto steps_before = [&](uint32_t at, Cursor& c) -> uint32_t {
            const uint32_t q = at / per_step;  // the sequence whose costs, of one item each, hold this
            uint32_t cost = 0, steps = 0, hit;
            Scan x = head;
            int b0 = 0;
            while (!(hit = __ballot_sync(0xffffffffu, cost + x.cost > q))) {
                cost += __shfl_sync(0xffffffffu, x.cost, 31);
                steps += __shfl_sync(0xffffffffu, x.steps, 31);
                b0 += 32;
                if (b0 >= all) return steps * per_step;  // the end
                x = scan_at<STEP, LIST>(a, cap, shared, b0);
            }
            const int f = __ffs(hit) - 1;
            c.b = b0 + f;
            c.len = __shfl_sync(0xffffffffu, x.len, f);
            const uint32_t n = __shfl_sync(0xffffffffu, x.n, f);
            cost += __shfl_sync(0xffffffffu, x.cost, f) - (n + kItemCost);
            steps += __shfl_sync(0xffffffffu, x.steps, f) - n;
            const uint32_t in_b = at - cost * per_step, item = in_b / (n + kItemCost), off = in_b - item * (n + kItemCost),
                           s = off < kItemCost ? 0 : off - kItemCost;
            c.n = (int)n;
            c.s = (int)s;
            c.kvh = (int)(item / (uint32_t)a.row_tiles);
            c.rt = (int)item - c.kvh * a.row_tiles;
            return steps * per_step + item * n + s;
        };
        const uint32_t first = steps_before(mine.first, cur);
        Cursor end;
        count = (int)(steps_before(mine.first + mine.count, end) - first);
        if (count == 0) return;
        cur.keys = keys_in<LIST>(a, cur.b, cur.len, shared);
    }

    // ---- the ring: this warp's keys of the steps ahead, whatever item they are of.  A key's row is D / 8 pieces of 16
    // bytes, piece c at c ^ (key % 8) (the lowest three bits), which keeps copies and ldmatrix free of bank conflicts.
    uint8_t* ring = smem + warp * C::RING;
    const uint32_t ring_u = smem_u32(ring);
    constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes per row, rows per copy instruction
    const int cr = lane / LPR, cc = lane % LPR;
    const __nv_bfloat16* kp = a.kp + cc * 8;
    const __nv_bfloat16* vp = a.vp + cc * 8;
    Cursor& ahead = sh.ahead[warp];  // the step to be looked up next; in shared memory to spare registers
    if (lane == 0) ahead = cur;
    __syncwarp();
    bool bad = false;
    // A step's keys are found in two loads that depend on each other (list, table), each a step ahead of its use.
    struct Keys {
        int tok, page, at;  // the lane's key: its token (kNone: none), logical page and place there
        int head, b;
    };
    int looked = 0, issued = 0;
    struct {
        int entry, off, len, kvh, b;  // the block list's entry for the lane's key, and the key's place in the block
    } from_list;
    Keys next;       // its page's entry of the table is loaded
    int next_entry;
    auto move_on = [&]() {
        if (++looked < count) {
            Cursor c = ahead;
            advance<STEP, LIST>(c, a, cap, shared);
            __syncwarp();
            if (lane == 0) ahead = c;
            __syncwarp();
        }
    };
    auto look_list = [&]() {  // LIST: the list's entries of step `looked`
        const int key = ahead.s * STEP + warp * KEYS + lane % KEYS;
        from_list.len = ahead.len;
        from_list.kvh = ahead.kvh;
        from_list.b = ahead.b;
        const int i = (int)a.block.div(key);
        from_list.off = key - i * (int)a.block.d;
        from_list.entry = looked < count && key < ahead.keys
                              ? a.list[((long long)ahead.b * a.Hkv + ahead.kvh) * a.keep + i]
                              : -1;
        move_on();
    };
    auto look_table = [&]() {  // the table's entries of the step after the one issued next
        if constexpr (LIST) {
            next.b = from_list.b;
            next.head = from_list.kvh;
            const int blocks = (int)a.block.div(from_list.len + a.block.d - 1);
            if (from_list.entry >= blocks) bad = true;
            next.tok = from_list.entry >= 0 && from_list.entry < blocks ? from_list.entry * (int)a.block.d + from_list.off : kNone;
            if (next.tok >= from_list.len) next.tok = kNone;
        } else {
            const int key = ahead.s * STEP + warp * KEYS + lane % KEYS;
            next.b = ahead.b;
            next.head = ahead.kvh;
            const bool prefix = ahead.b >= a.B;
            if (prefix) next.b = from;
            next.tok = looked < count && key < ahead.keys ? (prefix ? key : key + ahead.len - ahead.keys) : kNone;
        }
        const int lpage = next.tok == kNone ? 0 : (int)a.page.div(next.tok);
        next.at = next.tok - lpage * P;
        next_entry = next.tok == kNone ? -1 : a.table[(long long)next.b * a.max_pages + lpage];
        if (!LIST) move_on();
    };
    auto issue = [&](int slot) {
        if (issued < count) {
            const bool in = next.tok != kNone, ok = in && (unsigned)next_entry < (unsigned)a.num_pages;
            bad |= in && !ok;
            const uint32_t row = ok ? ((uint32_t)next_entry * a.Hkv + next.head) * P + next.at : ~0u;  // cache row
            const uint32_t base = ring_u + slot * C::SLOT;
            if (lane < KEYS) reinterpret_cast<int*>(ring + slot * C::SLOT + 2 * C::HALF)[lane] = next.tok;
#pragma unroll
            for (int n = 0; n < KEYS / RPI; ++n) {
                const int key = n * RPI + cr;
                const uint32_t rr = __shfl_sync(0xffffffffu, row, key);
                const bool there = rr != ~0u;
                const size_t off = (size_t)(there ? rr : 0u) * D;
                const uint32_t to = base + key * (D * 2) + ((cc ^ (key & 7)) << 4);
                copy16(to, kp + off, there);
                copy16(to + C::HALF, vp + off, there);
            }
        }
        ++issued;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // a step's keys are read by the warps of the group
    auto group_sync = [&]() {
        if constexpr (RG == 1)
            __syncwarp();
        else if (kg == 0)
            bar_sync(1, RG * 32);
        else
            bar_sync(2, RG * 32);
    };
    // ---- Q fragments: k-step s of lane (g, t): row g, columns 16 s + 2 t, + 1 and 16 s + 8 + 2 t, + 1
    uint32_t qb[NB][KS][2];
    auto load_q = [&]() {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            int r = cur.rt * ROWS + (rg * NB + nb) * 8 + g, b = cur.b;
            bool there = r < a.rows;
            if (!LIST && cur.b >= a.B) {  // row r of the prefix is row r % rows of sequence r / rows
                r += (cur.b - a.B) * ROWS;
                there = r < a.joint;
                b = there ? r / a.rows : 0;
                r -= b * a.rows;
            }
            const uint32_t* src =
                reinterpret_cast<const uint32_t*>(a.q + (((long long)b * a.Hkv + cur.kvh) * a.rows + (there ? r : 0)) * D) + t;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qb[nb][s][0] = there ? src[s * 8] : 0u;
                qb[nb][s][1] = there ? src[s * 8 + 4] : 0u;
            }
        }
    };
    if (LIST) look_list();
    look_table();
    if (LIST) look_list();
    load_q();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        issue(i);
        look_table();
        if (LIST) look_list();
    }

    // ---- the steps
    float acc[NB][D / 16][4];           // O^T: columns 16 i + g + 8 (c / 2) of rows 2 t + c % 2 of each eight
    float m[NB][2], l[NB][2];           // of rows 2 t + j; the references start at the lowest number: a row that sees no
                                        // key keeps l = 0 (2^(-inf - m))
    int seg = 0, slot = 0;              // first step of the segment within its item; ring slot
    bool begins = true;
    // fragment addresses: rows of the lane's part of ldmatrix, and its piece of 16 bytes
    const int kr = lane % 16, kc = lane / 16, vr = lane % 8 + lane / 16 * 8, vc = lane / 8 % 2;
    for (int it = 0; it < count; ++it) {
        const bool prefix = !LIST && cur.b >= a.B;
        const int r0 = cur.rt * ROWS + rg * NB * 8;                                           // of the warp
        const int nrows = min(ROWS, prefix ? a.joint - (cur.b - a.B) * ROWS : a.rows - cur.rt * ROWS);  // of the tile
        const long long bh = (long long)cur.b * a.Hkv + cur.kvh;
        if (begins) {
            seg = cur.s;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) acc[nb][i][0] = acc[nb][i][1] = acc[nb][i][2] = acc[nb][i][3] = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) m[nb][j] = -FLT_MAX, l[nb][j] = 0.f;
            }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        group_sync();  // every lane's copies are there, and the slot before is read
        issue(slot == 0 ? kStages - 1 : slot - 1);
        look_table();
        if (LIST) look_list();
        const int sees_all = cur.len - Nq;  // every row sees the tokens up to this one
        // A value product multiplies a key's V by the zero weights of the rows that do not see it, and 0 x infinity is NaN.
        // Where some rows see a key and others do not (the last Nq - 1 tokens), infinities and NaN are added to the sums of
        // the rows that do, and become zeros in the stage.
        if (DRAFTS && (LIST || (cur.s + 1) * STEP > cur.keys - Nq + 1)) {
            uint8_t* group = smem + kg * RG * C::RING + slot * C::SLOT;  // of key part * KEYS + k: + part * RING
            auto tok_of = [&](int key) {
                return reinterpret_cast<const int*>(group + key / KEYS * C::RING + 2 * C::HALF)[key % KEYS];
            };
            constexpr int WORDS = (RG * KEYS + 31) / 32;
            uint32_t partly[WORDS], any = 0;  // the keys that some rows see and others do not
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                const int tok = tok_of(min(w * 32 + lane, RG * KEYS - 1));
                any |= partly[w] = __ballot_sync(0xffffffffu, w * 32 + lane < RG * KEYS && tok > sees_all && tok != kNone);
            }
            auto each = [&](auto f) {
#pragma unroll
                for (int w = 0; w < WORDS; ++w)
#pragma unroll 1
                    for (uint32_t m = partly[w]; m; m &= m - 1) f(w * 32 + __ffs(m) - 1);
            };
            if (any) {
                auto word_of = [&](int key, int col) {  // the word of columns col, col + 1
                    return reinterpret_cast<uint32_t*>(group + key / KEYS * C::RING + C::HALF + key % KEYS * (D * 2) +
                                                       (((col / 8) ^ (key & 7)) << 4)) + col % 8 / 2;
                };
                auto wild = [](uint32_t half) { return (half & 0x7F80u) == 0x7F80u; };
                bool found = false;
                each([&](int key) {
                    for (int c = lane * 2; c < D; c += 64) {
                        const uint32_t w = *word_of(key, c);
                        found |= wild(w & 0xFFFFu) || wild(w >> 16);
                    }
                });
                if (__any_sync(0xffffffffu, found)) {  // in all warps of the group alike
                    each([&](int key) {
                        const int tok = tok_of(key);
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int col = 16 * i + g + 8 * h;
                                const uint32_t half = *word_of(key, col & ~1) >> (col & 1) * 16 & 0xFFFFu;
                                if (!wild(half)) continue;
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                    for (int j = 0; j < 2; ++j)
                                        if (tok <= sees_all + (r0 + nb * 8 + 2 * t + j) % Nq)
                                            acc[nb][i][2 * h + j] += __uint_as_float(half << 16);
                            }
                    });
                    group_sync();  // every warp has read them
                    each([&](int key) {
                        if (key / KEYS != rg) return;
                        for (int c = lane * 2; c < D; c += 64) {
                            uint32_t* w = word_of(key, c);
                            *w &= (wild(*w & 0xFFFFu) ? 0u : 0xFFFFu) | (wild(*w >> 16) ? 0u : 0xFFFF0000u);
                        }
                    });
                    group_sync();
                }
            }
        }
#pragma unroll 1
        for (int part = 0; part < RG; ++part) {
            if (cur.s * STEP + (kg * RG + part) * KEYS >= cur.keys || rg * NB * 8 >= nrows) break;
            const uint8_t* st = smem + (kg * RG + part) * C::RING + slot * C::SLOT;
            const uint32_t st_u = smem_u32(st);
            float S[NB][MT][4];  // keys 16 i + g, + 8 (c / 2) of rows 2 t + c % 2
            {
                float T[NB][MT][2][4] = {};  // two chains of products, which wait for each other half as often
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t ka[4];
                        ldmatrix4(ka, st_u + (i * 16 + kr) * (D * 2) + (((2 * s + kc) ^ (kr & 7)) << 4));
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_bf16(T[nb][i][s & 1], ka, qb[nb][s][0], qb[nb][s][1]);
                    }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) S[nb][i][c] = (T[nb][i][0][c] + T[nb][i][1][c]) * a.scale_log2;
            }
            const int* toks = reinterpret_cast<const int*>(st + 2 * C::HALF);
            const bool masked = (LIST || (cur.s + 1) * STEP > cur.keys - Nq + 1) &&
                                __any_sync(0xffffffffu, toks[lane % KEYS] > sees_all);
            uint32_t pb[NB][MT][2], pl[NB][MT][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                auto& x = S[nb];
                if (masked) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int tok = toks[i * 16 + h * 8 + g];
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (tok > sees_all + (DRAFTS ? (r0 + nb * 8 + 2 * t + j) % Nq : 0)) x[i][2 * h + j] = -INFINITY;
                        }
                }
                // softmax: m need not be the maximum, only within 2^8 of it: most steps find no larger one and skip the
                // reductions
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
                        const float f = ex2(fmaxf(m[nb][j] - top, -120.f));  // not 0: an infinite sum stays one
                        l[nb][j] *= f;
                        m[nb][j] = top;
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
                        const float p0 = ex2(x[i][2 * h] - m[nb][0]), p1 = ex2(x[i][2 * h + 1] - m[nb][1]);
                        l[nb][0] += p0;
                        l[nb][1] += p1;
                        const uint32_t hi = pack_bf16(p0, p1);
                        pb[nb][i][h] = transpose8x8(hi);
                        pl[nb][i][h] = transpose8x8(
                            pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u)));
                    }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t va[4];
                    ldmatrix4_trans(va, st_u + C::HALF + (i * 16 + vr) * (D * 2) + (((2 * c + vc) ^ (vr & 7)) << 4));
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        mma_bf16(acc[nb][c], va, pb[nb][i][0], pb[nb][i][1]);
                        mma_bf16(acc[nb][c], va, pl[nb][i][0], pl[nb][i][1]);
                    }
                }
        }
        slot = slot + 1 == kStages ? 0 : slot + 1;

        // ---- at the segment's end: O = sum over the warps with these rows of O_w 2^(m_w - m) / l
        const bool item_ends = cur.s + 1 == cur.n;
        begins = item_ends || it + 1 == count;
        const Cursor done = cur;
        if (it + 1 < count) advance<STEP, LIST>(cur, a, cap, shared);
        if (begins) {
            if (it + 1 < count) load_q();  // the next segment's queries come while this one's parts are joined
            float f[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], d);
                    const int r = nb * 8 + 2 * t + j;
                    if (g == 0) sh.stat[warp][0][r] = m[nb][j], sh.stat[warp][1][r] = l[nb][j];
                }
            sync();
            float* buf = reinterpret_cast<float*>(smem + C::MERGE) + g;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = nb * 8 + 2 * t + j;
                    float top = m[nb][j], sum = 0.f;
#pragma unroll
                    for (int w = 0; w < KG; ++w) top = fmaxf(top, sh.stat[w * RG + rg][0][r]);
#pragma unroll
                    for (int w = 0; w < KG; ++w) sum += sh.stat[w * RG + rg][1][r] * ex2(sh.stat[w * RG + rg][0][r] - top);
                    // a warp that saw none of the row's keys adds nothing (its V may have been infinite); NaN stays
                    f[nb][j] = l[nb][j] == 0.f ? 0.f : ex2(m[nb][j] - top) / sum;
                    if (l[nb][j] == 0.f)
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) acc[nb][i][j] = acc[nb][i][2 + j] = 0.f;
                    m[nb][j] = top;
                    l[nb][j] = sum;
                    if (kg > 0)
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                buf[((warp - RG) * 8 + 2 * t + j) * C::OROW + 16 * i + 8 * h] = acc[nb][i][2 * h + j] * f[nb][j];
                }
                sync();
                if (kg == 0) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float x = acc[nb][i][2 * h + j] * f[nb][j];
#pragma unroll
                                for (int w = 1; w < KG; ++w)
                                    x += buf[((w - 1) * RG + rg) * 8 * C::OROW + (2 * t + j) * C::OROW + 16 * i + 8 * h];
                                acc[nb][i][2 * h + j] = x;
                            }
                }
                if (nb + 1 < NB) sync();
            }
            if (kg == 0 && LIST && a.cluster) {  // into this CTA's shared memory, whose ring is done with
                float* to = reinterpret_cast<float*>(smem);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = (rg * NB + nb) * 8 + 2 * t + j;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            to[r * D + 16 * i + g] = acc[nb][i][j];
                            to[r * D + 16 * i + 8 + g] = acc[nb][i][2 + j];
                        }
                        if (g == 0) to[ROWS * D + r] = l[nb][j] == 0.f ? -INFINITY : m[nb][j] + lg2(l[nb][j]);
                    }
            } else if (kg == 0) {
                const bool whole = seg == 0 && item_ends && !prefix && (LIST || shared_of(shared, done.len, Nq) == 0);
                const long long item = bh * a.row_tiles + done.rt, slot_out = cta + item;
                if (tid == 0 && seg == 0) a.ends[2 * item] = cta;
                if (tid == 0 && item_ends) a.ends[2 * item + 1] = cta;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = (rg * NB + nb) * 8 + 2 * t + j;
                        if (r >= nrows) continue;
                        const float sum = l[nb][j], lse2 = sum == 0.f ? -INFINITY : m[nb][j] + lg2(sum);
                        if (whole) {
                            const long long row = bh * a.rows + done.rt * ROWS + r;  // (b, head, token) flattened
                            __nv_bfloat16* dst = a.o + row * D + g;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                dst[16 * i] = __float2bfloat16_rn(acc[nb][i][j]);
                                dst[16 * i + 8] = __float2bfloat16_rn(acc[nb][i][2 + j]);
                            }
                            if (a.lse && g == 0) a.lse[row] = lse2 * kLn2;
                        } else {
                            float* dst = a.part_o + (slot_out * ROWS + r) * D + g;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                dst[16 * i] = acc[nb][i][j];
                                dst[16 * i + 8] = acc[nb][i][2 + j];
                            }
                            if (g == 0) a.part_lse[slot_out * ROWS + r] = lse2;
                        }
                    }
            }
            sync();  // the statistics and buffers are read
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (LIST && a.cluster) {
        // the rows in turn to the cluster's CTAs: LSE = M + log2 sum 2^(lse_c - M), O = sum 2^(lse_c - M) o_c / sum
        float* mine = reinterpret_cast<float*>(smem);
        if (count == 0 && tid < ROWS) mine[ROWS * D + tid] = -INFINITY;
        if (a.cluster > 1) cluster_sync(); else __syncthreads();
        const int rank = blockIdx.x % a.cluster, bh = cur.b * a.Hkv + cur.kvh;
        constexpr int LANES = D / 4, AT_ONCE = kThreads / LANES;  // four columns of a row per thread
        const int col = tid % LANES * 4, nrows = min(ROWS, a.rows - cur.rt * ROWS);
        for (int r = rank * AT_ONCE + tid / LANES; r < nrows; r += a.cluster * AT_ONCE) {
            float lse[kMostCluster], M = -INFINITY, sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int c = 0; c < kMostCluster; ++c) {
                lse[c] = c < a.cluster ? ld_cluster_f32(smem_u32(mine + ROWS * D + r), c) : -INFINITY;
                M = fmaxf(M, lse[c]);
            }
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int c = 0; c < kMostCluster; ++c) {
                const float f = ex2(lse[c] - base);
                sum += f;
                if (c < a.cluster && f != 0.f) {  // a part without keys is nothing, whatever is in its place; NaN stays
                    const float4 x = ld_cluster_f4(smem_u32(mine + r * D + col), c);
                    o.x = fmaf(f, x.x, o.x);
                    o.y = fmaf(f, x.y, o.y);
                    o.z = fmaf(f, x.z, o.z);
                    o.w = fmaf(f, x.w, o.w);
                }
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const long long row = (long long)bh * a.rows + cur.rt * ROWS + r;
            *reinterpret_cast<uint2*>(a.o + row * D + col) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
            if (a.lse && col == 0) a.lse[row] = sum == 0.f ? -INFINITY : (M + lg2(sum)) * kLn2;
        }
        if (a.cluster > 1) cluster_sync();  // the others have read this CTA's
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_invalid(a.err, kSiteCacheTable, -1);
}

// A row's parts: `n` slots from `slot` on of the segments, `pn` from `pslot` on of the shared prefix.
struct Parts {
    long long slot, pslot;
    int n, pn;
    bool done;  // written already
};

// An item's segments are those of the CTAs from that of its first to that of its last step; CTA c's is in slot c + item.
template <bool LIST>
__host__ __device__ __forceinline__ Parts find_parts(const Params& a, int b, int kvh, int rt, int row) {
    const int item = (b * a.Hkv + kvh) * a.row_tiles + rt, cap = a.max_pages * (int)a.page.d;
    int shared = 0, place = 0;
    int2 pre = make_int2(0, -1);
    if constexpr (!LIST) {
        shared = clamp_len(*a.shared, cap);
        place = (b * a.rows + row) / a.pre_rows;
        place = a.joint ? place * a.Hkv + kvh : kvh * a.pre_tiles + place;
        pre = reinterpret_cast<const int2*>(a.pre_ends)[place];
    }
    const int2 own = reinterpret_cast<const int2*>(a.ends)[item];
    const int len = clamp_len(a.lens[b], cap);
    Parts x{0, 0, 0, 0, false};
    if (keys_of<LIST>(a, len, shared) > 0) {
        x.slot = (long long)own.x + item;
        x.n = own.y - own.x + 1;
    }
    // (a prefix kernel whose waits ran out may not have noted its items' ends)
    if (!LIST && shared_of(shared, len, a.Nq) > 0 && pre.x >= 0 && pre.x <= pre.y && pre.y < a.pre_workers) {
        x.pslot = pre.x + a.pre_item + place;
        x.pn = pre.y - pre.x + 1;
    }
    x.done = x.n == 1 && (LIST || shared_of(shared, len, a.Nq) == 0);  // as decode_rows decides it, parts of the prefix or not
    return x;
}

template <int D, int ROWS>
inline Params rows_params(const DecodeRowsLaunch& a) {
    Params p;
    p.q = (const __nv_bfloat16*)a.q;
    p.kp = (const __nv_bfloat16*)a.kp;
    p.vp = (const __nv_bfloat16*)a.vp;
    p.table = a.table;
    p.lens = a.lens;
    p.list = a.list;
    p.shared = a.shared;
    p.o = (__nv_bfloat16*)a.o;
    p.lse = a.lse;
    p.part_o = a.part_o;
    p.part_lse = a.part_lse;
    p.ends = a.ends;
    p.pre_ends = a.pre_ends;
    p.pre_o = a.pre_o;
    p.pre_lse = a.pre_lse;
    p.B = a.B;
    p.Hkv = a.Hkv;
    p.Nq = a.Nq;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.rows = a.Hq / a.Hkv * a.Nq;
    p.row_tiles = (p.rows + ROWS - 1) / ROWS;
    p.per_row = FastDiv((uint32_t)p.rows);
    p.heads = FastDiv((uint32_t)a.Hkv);
    p.keep = a.keep;
    p.pre_workers = a.pre_workers;
    p.pre_tiles = a.pre_tiles;
    p.pre_rows = a.pre_rows;
    p.pre_item = 0;
    p.joint = a.joint;
    p.tiles = (a.joint + ROWS - 1) / ROWS;
    if (a.joint) {  // its parts are among the others'
        p.pre_o = a.part_o;
        p.pre_lse = a.part_lse;
        p.pre_tiles = p.tiles;
        p.pre_rows = ROWS;
        p.pre_item = a.B * a.Hkv;
        p.pre_ends = a.ends + 2 * p.pre_item;
    }
    p.page = FastDiv((uint32_t)a.page);
    p.block = FastDiv((uint32_t)std::max(a.block, 1));
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    p.cluster = p.workers = 0;
    return p;
}

}  // namespace
}  // namespace fa
