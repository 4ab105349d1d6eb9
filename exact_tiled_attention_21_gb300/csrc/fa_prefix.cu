// Attention of a batch's new tokens over the prefix that all its sequences share,
// read once for all of them.
//
// The rows of all sequences (B x Hq / Hkv x Nq per kv head) against the prefix's
// keys are a dense product: per 256 rows and 128 keys 2 x 2 x 256 x 128 x d flops
// for 128 x 4 d bytes, so a batch of 64 sequences with 4 heads per kv head is as
// much bound by the tensor cores as by HBM, and fewer rows by HBM.  The keys come
// through the block table of the first sequence that has them all.
//
// GB300 mapping (one persistent CTA per SM, 320 threads, 512 TMEM columns), that of
// the forward: two 128-row tiles of queries share every key block.
//   warp 8      TMA producer of K and V through a ring of slots, in boxes of
//               R = gcd(page, 128) rows (a box never crosses a page), a lane each.
//   warp 9      MMA issuer: S_t = Q_t K^T into TMEM, O_t += P_t V with P_t read from
//               TMEM, the two tiles in turn (one only where there are up to 128
//               rows).
//   warps 0-3, 4-7   softmax of tile 0 and 1, thread = row; they also bring the
//               tile's query rows, which come from all sequences, into shared memory
//               and write the part of each row, O / l in fp32 and its LSE.
// Work: steps of 128 keys over (kv head, 256 rows), cut into equal shares for the
// CTAs, or an equal number of CTAs for each (kv head, 256 rows) where that costs a few
// steps at most: a second start of the pipeline and a second part to write cost four
// (64 sequences, 512 rows per kv head, 32768 tokens: 111 us against 106).  The part of
// a (kv head, 256 rows) that a CTA holds goes to the workspace at slot CTA + item, and
// the merge of fa_decode_rows.cu joins the parts with each sequence's own.  Rows of a
// sequence that does not see all of the prefix are computed and not written: its own
// pass takes all its keys.
//
// Up to 16 rows of a sequence and kv head (32 in small batches), in eights, the own
// tokens are this kernel's too: the
// prefix is bound by the tensor cores or, where it is short, by latencies, the own
// tokens by HBM, and run after one another they wait for each other's start and end.
// The CTAs are divided by the times that both would take; one with own tokens runs
// fa_decode_rows.cuh twice, on four warps each.  (32 sequences, 8192 shared tokens and up
// to 512 own ones, 4 heads per kv head: 31.3 us in two kernels, 23.7 in one; 64, 32768
// and 1000, two new tokens: 106 and 94.)  A pass over 16 or 32 rows at a time needs more
// registers than there are beside the prefix; the passes over eights read own tokens
// again, mostly out of L2.
#include <algorithm>

#include "fa_decode_rows.cuh"
#include "fa_softmax.cuh"

namespace fa {
namespace {

template <int D>
struct Pre {
    static constexpr int BN = 128, KCH = D / 64;
    static constexpr int Q_BYTES = 128 * D * 2, KV_BYTES = BN * D * 2, CHUNK = 128 * 128;
    static constexpr int NSLOT = D == 128 ? 5 : 8;
    static constexpr int OFF_Q = 0, OFF_KV = 2 * Q_BYTES;
    static constexpr int ROWS_BYTES = Cfg<D, 8>::SMEM, OFF_SHARED = 2 * ROWS_BYTES;  // the own tokens' two lots of four warps
    static constexpr int OFF_BAR = std::max(OFF_KV + NSLOT * KV_BYTES, OFF_SHARED + 2 * 1024);
    static_assert(sizeof(RowsShared<8>) <= 1024 && ROWS_BYTES % 128 == 0, "layout");
    // barriers: kv_full[NSLOT], kv_empty[NSLOT], q_full[2], s_full[3], p_full[3], o_final[2], pv_done, teardown.  s_full and
    // p_full: of tile 0's first buffer, of tile 1's, and of tile 0's second one where it is alone.  The last two share columns and not
    // a barrier: tile 1 passes over the segments of one tile, and a wait by parity is right only if none of a barrier's
    // earlier phases was passed over.
    static constexpr int NBAR = 2 * NSLOT + 12, OFF_MISC = OFF_BAR + NBAR * 8, SMEM = OFF_MISC + 16 + 1024;
    static constexpr int THREADS = 320;
    static constexpr uint32_t TMEM_COLS = 512, COL_S = 0, COL_O = 256;  // tile t: + 128 t, + D t
    static constexpr uint32_t IDESC_S = idesc_bf16(128, BN, 0, 0);      // Q, K both K-major
    static constexpr uint32_t IDESC_O = idesc_bf16(128, D, 0, 1);       // P from TMEM, V MN-major
    static_assert(SMEM <= 232448, "shared memory budget");
};

// What a CTA's second (kv head, tile of rows) costs, in steps: queries, a start of the pipeline and a part to write.
constexpr uint32_t kCrossing = 4;

// What the CTAs are divided by, in microseconds, from timings of nine batches at eight to twenty divisions each (64 sequences,
// 4096 shared tokens and up to 1000 own ones: 83.7 us with 8 CTAs for the prefix, 41.9 with 32, 51.1 with 64, 132 with 128): a
// step of the prefix, of one tile and of two, how much later a CTA's first is done than one of own tokens, and a second item;
// of own tokens, a step of four warps, and an item's start and end, both beside a prefix.  The times are within a tenth of
// the best division's.
template <int D, int OWN>
struct Times {
    static constexpr float ONE_STEP = D == 128 ? 0.92f : 0.75f, TWO_STEP = D == 128 ? 1.8f : 1.45f;
    static constexpr float ONE_START = 5.f, TWO_START = D == 128 ? 9.f : 5.f, CROSSING = 6.5f;
    static constexpr float OWN_STEP = D == 64 ? 1.1f : OWN == 2 ? 1.45f : 1.2f, OWN_ITEM = D == 64 ? 1.6f : 2.5f;
};

struct PreParams {
    const __nv_bfloat16* q;
    const int* table;   // int32 [B, max_pages]
    const int* lens;
    const int* shared;  // [1]
    float* part_o;      // [slot][tile_rows][D]
    float* part_lse;    // [slot][tile_rows], log2
    int* ends;          // [item][2]: the CTAs of its first and last step
    int B, Hkv, Nq, rows, page, max_pages, num_pages, tiles, tile_rows, box;
    FastDiv per_row;  // rows
    float scale_log2;
    DevError* err;
    uint64_t timeout_ns;
};

template <int D, int OWN>
__global__ void __launch_bounds__(Pre<D>::THREADS, 1)
prefix_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const PreParams p,
              const __grid_constant__ Params own) {
    using C = Pre<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t s_base = smem_u32(smem), bar0 = s_base + C::OFF_BAR;
    auto bar_full = [&](int s) { return bar0 + 8 * s; };
    auto bar_empty = [&](int s) { return bar0 + 8 * C::NSLOT + 8 * s; };
    const uint32_t BAR_Q = bar0 + 16 * C::NSLOT, BAR_S = BAR_Q + 16, BAR_P = BAR_S + 24, BAR_O = BAR_P + 24, BAR_PV = BAR_O + 16,
                   BAR_TD = BAR_PV + 8;
    uint32_t* tmem_slot = (uint32_t*)(smem + C::OFF_MISC);
    volatile int* abort_flag = (volatile int*)(smem + C::OFF_MISC + 4);
    const WaitCtl ctl{p.err, p.timeout_ns, abort_flag};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        *abort_flag = 0;
        for (int s = 0; s < 2 * C::NSLOT; ++s) mbar_init(bar0 + 8 * s, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(BAR_Q + 8 * t, 128);
            mbar_init(BAR_O + 8 * t, 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(BAR_S + 8 * i, 1);
            mbar_init(BAR_P + 8 * i, 128);
        }
        mbar_init(BAR_PV, 1);
        mbar_init(BAR_TD, 1);
        fence_mbar_init();
        if ((s_base & 1023u) != 0) record_error(ctl, kErrTimeout, kSiteAlign, (int)(s_base & 1023u));
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    const int cap = p.max_pages * p.page, given = *p.shared, shared = min(max(given, 0), cap);
    if (blockIdx.x == 0) check_lengths(p.lens, OWN > 0 ? p.B : 0, cap, given, p.err);
    int from = -1;  // the first sequence that sees all of the prefix
    for (int b0 = 0; b0 < p.B && from < 0; b0 += 32) {
        const uint32_t hit = __ballot_sync(0xffffffffu, b0 + lane < p.B && min(max(p.lens[min(b0 + lane, p.B - 1)], 0), cap) - p.Nq >= shared);
        if (hit) from = b0 + __ffs(hit) - 1;
    }
    const uint32_t steps = from < 0 ? 0 : (uint32_t)(shared + 127) / 128;  // of an item, a (kv head, tile of rows)
    const uint32_t items = (uint32_t)p.Hkv * p.tiles;
    uint32_t ctas = gridDim.x;  // of the prefix; the others have the own tokens
    if constexpr (OWN > 0) {
        using T = Times<D, OWN>;
        const uint2 cost = cost_of_all<Cfg<D, 8>::STEP, false>(own, cap, shared);  // of one kv head's items: steps and costs
        const float each = (float)(own.Hkv * own.row_tiles),
                    rest = each * (T::OWN_STEP * (float)cost.x + T::OWN_ITEM * (float)(cost.y - cost.x));
        const float step = p.tile_rows > 128 ? T::TWO_STEP : T::ONE_STEP, start = p.tile_rows > 128 ? T::TWO_START : T::ONE_START;
        // a lane has two divisions to compare: n CTAs, the same number for each item, and fewer than items
        const uint32_t most = (gridDim.x - 1) / items, few = min(items, gridDim.x);
        const uint32_t k = (lane + 1) * most / 32, n0 = k * items, n1 = max((lane + 1) * few / 33, 1u);
        const float time0 = k ? fmaxf(start + step * ceilf(__fdividef((float)steps, (float)k)), __fdividef(rest, (float)(2 * (gridDim.x - n0))))
                              : FLT_MAX,
                    time1 = fmaxf(start + __fdividef((float)items, (float)n1) * (step * (float)steps + T::CROSSING),
                                  __fdividef(rest, (float)(2 * (gridDim.x - n1))));
        const uint32_t mine = __float_as_uint(fminf(time0, time1)), least = __reduce_min_sync(0xffffffffu, mine);
        ctas = steps ? __reduce_min_sync(0xffffffffu, mine == least ? (time0 <= time1 ? n0 : n1) : ~0u) : 0;
    }
    const uint32_t per = ctas / items;
    Share mine = {0, 0};
    if (per && (steps + per - 1) / per <= (steps * items + ctas - 1) / ctas + kCrossing) {  // `per` CTAs for each item
        const uint32_t item = blockIdx.x / per;
        if (item < items) mine = share_of(steps, per, blockIdx.x - item * per);
        mine.first += item * steps;
    } else if (blockIdx.x < ctas) {
        mine = share_of(steps * items, ctas, blockIdx.x);
    }
    const uint32_t u0 = mine.first, u1 = u0 + mine.count, c = blockIdx.x;
    const int all = p.B * p.rows;  // rows of a kv head
    // one role's walk over the CTA's segments: item, its steps [s0, s1)
    struct Segment {
        int item, kvh, row0, s0, s1;
        bool two;  // more than 128 rows
    };
    auto segment_at = [&](uint32_t u) {
        Segment g;
        g.item = (int)(u / steps);
        g.s0 = (int)(u - g.item * steps);
        g.s1 = (int)min(steps, g.s0 + (u1 - u));
        g.kvh = g.item / p.tiles;
        g.row0 = (g.item - g.kvh * p.tiles) * p.tile_rows;
        g.two = min(p.tile_rows, all - g.row0) > 128;
        return g;
    };

    if (OWN > 0 && blockIdx.x >= ctas) {
        // ------------------------------------------------------------ own tokens
        if (warp < 8) {
            const int half = warp >> 2;
            decode_rows<D, 8, OWN == 2, false, true>(own, smem + half * C::ROWS_BYTES,
                                                     reinterpret_cast<RowsShared<8>*>(smem + C::OFF_SHARED)[half], tid & 127,
                                                     2 * (blockIdx.x - ctas) + half, 2 * (gridDim.x - ctas), 1 + half);
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------ TMA producer (whole warp)
        const uint64_t policy = l2_policy_evict_first();
        if (lane == 0) {
            tma_prefetch_desc(&map_k);
            tma_prefetch_desc(&map_v);
        }
        const int R = p.box;
        int slot = 0;
        uint32_t phase = 0, issued = 0, issued_par = 0;
        bool ok = !*abort_flag;
        // the page of the lane's box of a step, loaded one step ahead
        auto page_of = [&](const Segment& g, int s) {
            const int key = s * 128 + lane * R;
            return lane * R < 128 && key < shared ? p.table[(long long)from * p.max_pages + key / p.page] : 0;
        };
        int pg_next = 0;
        if (u0 < u1) {
            const Segment g = segment_at(u0);
            pg_next = page_of(g, g.s0);
        }
        for (uint32_t u = u0; u < u1 && ok;) {
            const Segment g = segment_at(u);
            for (int s = g.s0; s < g.s1 && ok; ++s, ++u) {
                const int nk = min(128, shared - s * 128), nbox = (nk + R - 1) / R;
                int pg = pg_next;
                if (u + 1 < u1) pg_next = page_of(g, s + 1 < (int)steps ? s + 1 : 0);
                const int key = s * 128 + lane * R, row = key - key / p.page * p.page;
                if (lane < nbox && (unsigned)pg >= (unsigned)p.num_pages) {
                    record_invalid(p.err, kSitePagedTable, pg);
                    pg = p.num_pages;  // wholly out of range: zero fill
                }
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    if (lane == 0) {
                        ok = mbar_wait(bar_empty(slot), phase ^ 1, ctl, kSiteKvEmpty);
                        if (ok) mbar_arrive_expect_tx(bar_full(slot), (uint32_t)(nbox * R * D * 2));
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane < nbox) {
                        const uint32_t dst = s_base + C::OFF_KV + slot * C::KV_BYTES + (uint32_t)(lane * R * 128);
                        for (int h = 0; h < C::KCH; ++h)
                            tma_load_4d(dst + h * C::CHUNK, kv ? &map_v : &map_k, bar_full(slot), h * 64, row, g.kvh, pg, policy);
                    }
                    issued |= 1u << slot;
                    issued_par = (issued_par & ~(1u << slot)) | (phase << slot);
                    if (++slot == C::NSLOT) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        if (lane == 0 && *abort_flag)  // let every load in flight land before the CTA exits
            for (int s = 0; s < C::NSLOT; ++s)
                if (issued & (1u << s)) mbar_drain(bar_full(s), (issued_par >> s) & 1, ctl, kSiteTeardown);
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && !*abort_flag) {
            int slot = 0;
            uint32_t phase = 0, p_iter = 0, q_iter = 0, p1_iter = 0, p2_iter = 0, q1_iter = 0;
            auto issue_s = [&](int t, uint32_t sK, int buf) {
                const uint64_t a0 = sdesc_sw128(s_base + C::OFF_Q + t * C::Q_BYTES, 16, 1024), b0 = sdesc_sw128(sK, 16, 1024);
                const uint32_t d = tmem + C::COL_S + 128 * buf;
                mma_ss_first(d, a0, b0, C::IDESC_S);
#pragma unroll
                for (int k = 1; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * C::CHUNK + (k & 3) * 32;
                    mma_ss_acc(d, sdesc_add(a0, off), sdesc_add(b0, off), C::IDESC_S);
                }
            };
            auto issue_o = [&](int t, uint32_t sV, bool acc, int buf) {
                const uint64_t b0 = sdesc_sw128(sV, C::CHUNK, 1024);
                const uint32_t d = tmem + C::COL_O + D * t, pc = tmem + C::COL_S + 128 * buf;
                mma_ts(d, pc, b0, C::IDESC_O, acc ? 1u : 0u);
#pragma unroll
                for (int k = 1; k < C::BN / 16; ++k) mma_ts_acc(d, pc + k * 8, sdesc_add(b0, k * 2048), C::IDESC_O);
            };
            auto next = [&]() {
                if (++slot == C::NSLOT) {
                    slot = 0;
                    phase ^= 1;
                }
            };
            auto kv_at = [&](int s) { return s_base + C::OFF_KV + s * C::KV_BYTES; };
            bool ok = true;
            for (uint32_t u = u0; u < u1 && ok;) {
                const Segment g = segment_at(u);
                if (!mbar_wait(BAR_Q, q_iter++ & 1, ctl, kSiteQFull)) break;
                if (g.two && !mbar_wait(BAR_Q + 8, q1_iter++ & 1, ctl, kSiteQFull)) break;
                int kslot = slot;
                if (!mbar_wait(bar_full(kslot), phase, ctl, kSiteKvFull)) break;
                tc_fence_after();
                next();
                issue_s(0, kv_at(kslot), 0);
                mma_commit(BAR_S);
                if (!g.two) {
                    // one tile: the scores of the next block, into the other tile's columns, before the product of this one
                    mma_commit(bar_empty(kslot));
                    for (int s = g.s0; s < g.s1; ++s, ++u) {
                        const int buf = (s - g.s0) & 1, vslot = slot;
                        const uint32_t vphase = phase;
                        next();
                        if (s + 1 < g.s1) {
                            kslot = slot;
                            if (!mbar_wait(bar_full(kslot), phase, ctl, kSiteKvFull)) { ok = false; break; }
                            tc_fence_after();
                            next();
                            issue_s(0, kv_at(kslot), buf ^ 1);
                            mma_commit(BAR_S + 16 * (buf ^ 1));
                            mma_commit(bar_empty(kslot));
                        }
                        if (!mbar_wait(bar_full(vslot), vphase, ctl, kSiteKvFull)) { ok = false; break; }
                        if (!mbar_wait(BAR_P + 16 * buf, (buf ? p2_iter++ : p_iter++) & 1, ctl, kSitePFull)) { ok = false; break; }
                        tc_fence_after();
                        issue_o(0, kv_at(vslot), s > g.s0, buf);
                        mma_commit(bar_empty(vslot));
                        mma_commit(s + 1 < g.s1 ? BAR_PV : BAR_O);
                    }
                    continue;
                }
                issue_s(1, kv_at(kslot), 1);
                mma_commit(BAR_S + 8);
                mma_commit(bar_empty(kslot));
                for (int s = g.s0; s < g.s1; ++s, ++u) {
                    const bool more = s + 1 < g.s1;
                    const int vslot = slot;
                    if (!mbar_wait(bar_full(vslot), phase, ctl, kSiteKvFull)) { ok = false; break; }
                    next();
                    if (!mbar_wait(BAR_P, p_iter++ & 1, ctl, kSitePFull)) { ok = false; break; }
                    tc_fence_after();
                    issue_o(0, kv_at(vslot), s > g.s0, 0);
                    if (more) {
                        kslot = slot;
                        if (!mbar_wait(bar_full(kslot), phase, ctl, kSiteKvFull)) { ok = false; break; }
                        tc_fence_after();
                        next();
                        issue_s(0, kv_at(kslot), 0);
                        mma_commit(BAR_S);
                    } else {
                        mma_commit(BAR_O);
                    }
                    if (!mbar_wait(BAR_P + 8, p1_iter++ & 1, ctl, kSitePFull)) { ok = false; break; }
                    tc_fence_after();
                    issue_o(1, kv_at(vslot), s > g.s0, 1);
                    mma_commit(bar_empty(vslot));
                    if (more) {
                        issue_s(1, kv_at(kslot), 1);
                        mma_commit(BAR_S + 8);
                        mma_commit(bar_empty(kslot));
                    } else {
                        mma_commit(BAR_O + 8);
                    }
                }
            }
            if (*abort_flag) {  // every MMA issued so far must finish before TMEM is freed
                mma_commit(BAR_TD);
                mbar_drain(BAR_TD, 0, ctl, kSiteTeardown);
            }
        }
    } else {
        // ------------------------------------------------------------ queries, softmax, epilogue
        const int t = warp >> 2, r = tid & 127;  // tile; row within it = TMEM lane
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t col_o = C::COL_O + D * t;
        // handoffs before the segment: by the three barriers of scores, of the products of one tile, of the ring's fills; of O so far
        uint32_t s_next0 = 0, s_next1 = 0, s_next2 = 0, pv_next = 0, kv_fill = 0, o_iter = 0;
        uint64_t skipped = 0;  // steps of one tile since tile 1's last segment
        for (uint32_t u = u0; u < u1;) {
            const Segment g = segment_at(u);
            const int nst = g.s1 - g.s0;
            u += nst;
            const uint32_t fill0 = kv_fill, s0 = s_next0, s1 = g.two ? s_next1 : s_next2, pv0 = pv_next;
            kv_fill += 2 * nst;
            s_next0 += g.two ? nst : (nst + 1) / 2;
            s_next1 += g.two ? nst : 0;
            s_next2 += g.two ? 0 : nst / 2;
            pv_next += g.two ? 0 : nst - 1;
            if (t == 1 && !g.two) {
                skipped += nst;
                continue;
            }
            // ---- the tile's query rows, coalesced: D / 8 lanes a row; those past the last one are zeros
            {
                uint8_t* sq = smem + C::OFF_Q + t * C::Q_BYTES;
                constexpr int LPR = D / 8, N = LPR;  // N rows of a thread, all in flight: the keys' copies fill the memory's queues
                const int piece = r % LPR, row = r / LPR;
                uint4 x[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int at = g.row0 + t * 128 + row + i * (128 / LPR);
                    const int b = (int)p.per_row.div(at);
                    x[i] = at < all ? *reinterpret_cast<const uint4*>(
                                          p.q + (((long long)b * p.Hkv + g.kvh) * p.rows + (at - b * p.rows)) * D + piece * 8)
                                    : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int to = row + i * (128 / LPR);
                    *reinterpret_cast<uint4*>(sq + (piece >> 3) * C::CHUNK + to * 128 + (((piece & 7) ^ (to & 7)) << 4)) = x[i];
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(BAR_Q + 8 * t);
            }
            float m_use = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < nst; ++j) {
                const int buf = g.two ? t : j & 1;  // one tile takes both buffers in turn
                const uint32_t col_s = C::COL_S + 128 * buf, bar = 8 * (g.two ? t : 2 * buf);
                const uint32_t nth = (buf ? s1 : s0) + (g.two ? j : j >> 1);
                WaitCtl limit = ctl;  // tile 1's first scores come behind the segments that it passed over: 10 us a step
                limit.timeout_ns += skipped * 10000;
                skipped = 0;
                if (!mbar_wait(BAR_S + bar, nth & 1, limit, kSiteSFull)) { ok = false; break; }
                tc_fence_after();
                const int nk = min(128, shared - (g.s0 + j) * 128);  // at least 1
                const float mraw = nk < 128 ? row_max_pass<true>(lane_addr + col_s, nk - 1, 0)
                                            : row_max_pass<false>(lane_addr + col_s, 127, 0);
                const float m_new = fmaxf(m_use, mraw * p.scale_log2);
                if (j == 0) {
                    m_use = m_new;
                } else if (__any_sync(0xffffffffu, m_new > m_use + 8.f)) {
                    // rescale the accumulator so that O and l keep a common reference; with one tile the product before
                    // may still be running
                    if (!g.two) {
                        if (!mbar_wait(BAR_PV, (pv0 + j - 1) & 1, ctl, kSitePFull)) { ok = false; break; }
                        tc_fence_after();
                    }
                    const float alpha = m_new == -INFINITY ? 1.f : ex2(m_use - m_new);
#pragma unroll 1
                    for (int q4 = 0; q4 < D / 32; ++q4) {
                        uint32_t v[32];
                        tmem_ld32(lane_addr + col_o + q4 * 32, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                        tmem_st32(lane_addr + col_o + q4 * 32, v);
                    }
                    l *= alpha;
                    m_use = m_new;
                }
                const float msub = m_use == -INFINITY ? 0.f : m_use;
                l += nk < 128 ? exp_pass<true>(lane_addr + col_s, lane_addr + col_s, nk - 1, 0, p.scale_log2, msub)
                              : exp_pass<false>(lane_addr + col_s, lane_addr + col_s, 127, 0, p.scale_log2, msub);
                if (nk < 128 && t == 0) {  // V rows past the prefix may hold anything: zeros, since 0 x NaN would not vanish.
                                           // Tile 1's product follows tile 0's, which waits for this.
                    const uint32_t f = fill0 + 2 * j + 1;
                    if (!mbar_wait(bar_full(f % C::NSLOT), (f / C::NSLOT) & 1, ctl, kSiteKvFull)) { ok = false; break; }
                    if (r >= nk) {
                        uint4* row = reinterpret_cast<uint4*>(smem + C::OFF_KV + (f % C::NSLOT) * C::KV_BYTES + r * 128);
#pragma unroll
                        for (int h = 0; h < C::KCH; ++h)
#pragma unroll
                            for (int i = 0; i < 8; ++i) row[h * (C::CHUNK / 16) + i] = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                tc_fence_before();
                mbar_arrive(BAR_P + bar);
            }
            if (!ok || !mbar_wait(BAR_O + 8 * t, o_iter & 1, ctl, kSiteOFinal)) break;
            ++o_iter;
            tc_fence_after();
            // ---- the part of each row whose sequence sees the whole prefix
            const int at = g.row0 + t * 128 + r, b = at < all ? (int)p.per_row.div(at) : 0;
            const bool valid = at < all && min(max(p.lens[b], 0), cap) - p.Nq >= shared;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long place = (long long)(c + g.item) * p.tile_rows + t * 128 + r;
            if (tid == 0 && g.s0 == 0) p.ends[2 * g.item] = c;
            if (tid == 0 && g.s1 == (int)steps) p.ends[2 * g.item + 1] = c;
            float* dst = p.part_o + place * D;
#pragma unroll 1
            for (int q4 = 0; q4 < D / 32; ++q4) {
                uint32_t v[32];
                tmem_ld32(lane_addr + col_o + q4 * 32, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * inv);
                if (valid)
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + q4 * 32 + i), "r"(v[i]),
                                     "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]),
                                     "r"(v[i + 7])
                                     : "memory");
            }
            if (valid) p.part_lse[place] = l == 0.f ? -INFINITY : m_use + lg2(l);
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) {
        __syncwarp();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int D, int OWN>
cudaError_t launch_o(const PrefixLaunch& a, const DecodeRowsLaunch& rows, cudaStream_t s) {
    using C = Pre<D>;
    cudaError_t e = set_smem_limit_once<prefix_kernel<D, OWN>>(C::SMEM);
    if (e != cudaSuccess) return e;
    PreParams p;
    p.q = (const __nv_bfloat16*)a.q;
    p.table = a.table;
    p.lens = a.lens;
    p.shared = a.shared;
    p.part_o = a.part_o;
    p.part_lse = a.part_lse;
    p.ends = a.ends;
    p.B = a.B;
    p.Hkv = a.Hkv;
    p.Nq = a.Nq;
    p.rows = a.Hq / a.Hkv * a.Nq;
    p.page = a.page;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.tiles = a.tiles;
    p.tile_rows = a.tile_rows;
    p.box = a.box;
    p.per_row = FastDiv((uint32_t)p.rows);
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.err = a.err;
    p.timeout_ns = a.timeout_ns;
    return launch_dependent(prefix_kernel<D, OWN>, dim3((unsigned)a.workers), dim3(C::THREADS), C::SMEM, s, a.map_k, a.map_v, p,
                            rows_params<D, 8>(rows));
}

template <int D>
cudaError_t launch_d(const PrefixLaunch& a, const DecodeRowsLaunch& rows, cudaStream_t s) {
    if (!a.own) return launch_o<D, 0>(a, rows, s);
    return a.Nq == 1 ? launch_o<D, 1>(a, rows, s) : launch_o<D, 2>(a, rows, s);
}

}  // namespace

cudaError_t launch_prefix(const PrefixLaunch& a, const DecodeRowsLaunch& rows, cudaStream_t s) {
    return a.d == 128 ? launch_d<128>(a, rows, s) : launch_d<64>(a, rows, s);
}

}  // namespace fa
