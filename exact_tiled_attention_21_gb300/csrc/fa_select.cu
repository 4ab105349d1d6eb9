// Selection of the blocks of a paged cache that a query is likely to attend to.
//
// From the bounds that the append keeps of every block (the smallest and the
// largest key element of each column), a row q cannot score more with any key of
// block j than
//     u_j = sum_c max(q_c, 0) max_jc + min(q_c, 0) min_jc,
// and a block's score is the largest u_j of the kv head's query rows.  The first
// blocks, the most recent ones and, of the others, those of largest score stay.
//
// The scores are products on the tensor cores (mma.sync m16n8k16: 16 blocks, 8
// rows, the bounds as they come from memory, q split into its two parts), four
// chains of sums per block and row: with fp32 FMAs, of which a row needs 2 d per
// block, and sums over lanes the instructions took ten times as long as the bytes.
//
// The choice is that of exact scores.  The products of bf16 numbers are exact; a
// step adds 16 of them to a sum, off by at most 17 x 2^-24 of the largest term even
// if each is cut to 24 bits, and a chain has 2 d / 64 steps: the score is within E
// = 2^-17.9 A, with A the largest sum of |q_c| |bound_c| a row can have, bounded
// by 8 columns at a time.  Blocks further than 2 E from the smallest score that
// stays are decided; if the others do not all stay, theirs are summed again in whole
// numbers of 2^-61 A (off by 2^-58 A at most; in fp64 where something is not finite or
// tiny), and equal ones go by index.  One element of q or the bounds that is not finite leaves
// every block of its (sequence, kv head) to fp64: 5.0 ms for 4096 blocks, 0.64 ms for 256 of
// each of 32 sequences (d = 128, 4 rows, 8 kv heads); more than 256 undecided blocks without that
// are slower too (pages all alike: 131 us in place of 18, 25 in place of 14).
//
// 4 d bytes per block and 4 d flops per block and row.  Where contexts are long the bounds'
// way through shared memory and the queries' fragments, read again for every 16 blocks, bind it (32
// sequences of up to 16384 tokens, blocks of 16, 8 kv heads, d = 128: 27.5 us, 14.5 at the
// copy rate; DRAM below half of its peak under the profiler, short_scoreboard on top), otherwise
// latency (of 4096 tokens 12.9 us: 2 to the queries' fragments, 7 to the scores, which the
// first loads of all SMs at once take half of, 3.6 to the choice).  One
// cluster of up to 8 CTAs per (sequence, kv head) makes the scores, in the shared memory
// of its first CTA (or in the workspace), which chooses: a histogram over the scores'
// range finds the bin that the smallest one that stays is in, and counting greater
// ones within that bin finds it.
#include <algorithm>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kRowTile = 64;      // query rows in shared memory at once
constexpr int kBatch = 16;        // blocks of a warp's batch
constexpr int kBins = 1024, kList = 256;
constexpr float kError = 4e-6f;   // E / A: 2^-17.9

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// 16 bytes into shared memory; zeros if !ok (src must still be a valid address).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
// Largest magnitudes of the two halves of bf16 pairs, as bits: infinities and NaN on top.
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7FFF7FFFu));
    return r;
}

// The negative (or positive) elements of a pair of bf16, zeros in the others' places; NaN stays.
__device__ __forceinline__ uint32_t part2(uint32_t w, bool negative) {
    auto keep = [&](uint32_t h) { return ((h >> 15) != 0) == negative || (h & 0x7FFFu) > 0x7F80u; };
    return (keep(w & 0xFFFFu) ? w & 0xFFFFu : 0u) | (keep(w >> 16) ? w & 0xFFFF0000u : 0u);
}
__device__ __forceinline__ float abs_sum2(uint32_t w) {
    return fabsf(__uint_as_float(w << 16)) + fabsf(__uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Integers whose order is the numbers', -0 = +0; of a double also NaN, above everything.
__device__ __forceinline__ uint32_t key32(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t key64(double x) {
    if (x != x) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : u | (1ull << 63);
}

struct SelectPlan {
    int ctas;          // of a cluster
    int tiles;         // of 8 query rows in shared memory at once
    FastDiv per_page;  // blocks of a page
};

// Score of a row and a block in fp64, by 8 lanes; its key.  On its own: it is called where something is not finite, or tiny.
__device__ __noinline__ uint64_t slow_key(const __nv_bfloat16* q, const __nv_bfloat16* ends, int d, int part) {
    double sum = 0.0;
    for (int c = part; c < d; c += 8) {
        const double x = (double)__bfloat162float(q[c]);
        sum += (x > 0.0 ? 0.0 : x) * (ends ? (double)__bfloat162float(ends[c]) : 0.0) +
               (x < 0.0 ? 0.0 : x) * (ends ? (double)__bfloat162float(ends[d + c]) : 0.0);
    }
    for (int m = 1; m < 8; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    return key64(sum);
}

// GLOBAL: the scores go through the workspace (too many of them, or several tiles of query rows).  THREADS: 512 where a CTA
// has an SM to itself.
template <int D, bool GLOBAL, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) select_blocks_kernel(const SelectLaunch a, const SelectPlan plan) {
    constexpr int kSelThreads = THREADS, kSelWarps = THREADS / 32;
    constexpr int S = D / 16, CHUNKS = 4 * S;  // 64-byte pieces of a block's bounds, a lane's part of which is a chunk
    extern __shared__ __align__(16) uint4 s_mem[];
    // With 256 threads the next batch comes through shared memory while this one is worked on, a thread's pieces in places of its
    // own (32 sequences of up to 16384 tokens, blocks of 16: 39.3 us without, 33.0 with; 4096 tokens 15.9 and 14.3).  With 512
    // and an SM to itself a CTA has all its loads in flight anyway (one sequence of 131072 tokens: 16.4 without, 17.7 with).
    constexpr bool RING = THREADS == 256;
    uint4* s_ring = s_mem + threadIdx.x;                 // [2 S][THREADS]
    uint4* s_q = s_mem + (RING ? 2 * S * THREADS : 0);  // [tile of 8 rows][piece][lane]: B fragments of two products
    uint32_t* s_keys = reinterpret_cast<uint32_t*>(s_q + plan.tiles * S * 32);
    // bits of the largest sum of |q|, and |bound|, of each chunk; behind these the complement of the smallest key and the largest
    __shared__ uint32_t s_sum8[CHUNKS], s_big[CHUNKS + 2];
    __shared__ int s_hist[kBins];
    __shared__ uint64_t s_exact[kList];
    __shared__ uint32_t s_list[kList];
    __shared__ int2 s_sum[2][kSelWarps];
    __shared__ int s_found[2], s_many;
    __shared__ uint32_t s_key;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % plan.ctas;
    const int bh = blockIdx.x / plan.ctas, b = bh / a.Hkv, kvh = bh - b * a.Hkv;
    const int bpp = (int)plan.per_page.d, cap = a.max_pages * bpp * a.block;
    int len = a.lens[b];
    const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + (long long)bh * a.rows * D;
    // the B fragments of query rows [r0, r0 + many): a lane's chunk is 8 columns of a row's negative part (times the
    // smallest keys), then of its positive part
    auto stage = [&](int r0, int many) {
        for (int i = tid; i < (many + 7) / 8 * S * 32; i += kSelThreads) {
            const int l = i % 32, s = i / 32 % S, r = i / 32 / S * 8 + l / 4, chunk = s * 4 + l % 4;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (r < many) w = *reinterpret_cast<const uint4*>(q + (long long)(r0 + r) * D + chunk * 8 % D);
            const bool neg = chunk * 8 < D;
            w = make_uint4(part2(w.x, neg), part2(w.y, neg), part2(w.z, neg), part2(w.w, neg));
            s_q[i] = w;
            // rounded up: a sum of eight is off by 2^-21 at most
            const float sum = (abs_sum2(w.x) + abs_sum2(w.y) + abs_sum2(w.z) + abs_sum2(w.w)) * 1.00001f;
            atomicMax(&s_sum8[chunk], __float_as_uint(sum) & 0x7FFFFFFFu);
        }
    };
    if (tid < CHUNKS) s_sum8[tid] = 0;
    if (tid < CHUNKS + 2) s_big[tid] = 0;
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
    if (tid == 0) s_many = 0;
    __syncthreads();
    stage(0, min(kRowTile, a.rows));  // while the length comes
    if (len < 0 || len > cap) {
        if (tid == 0 && rank == 0) record_invalid(a.err, kSiteCacheLen, len);
        len = min(max(len, 0), cap);
    }
    const int n = (len + a.block - 1) / a.block;
    int* out = a.out + (long long)bh * a.keep;
    if (n <= a.keep) {  // all of them; the whole cluster alike
        if (rank == 0)
            for (int i = tid; i < a.keep; i += kSelThreads) out[i] = i < n ? i : -1;
        return;
    }
    const int j0 = a.first, mid = n - a.recent - j0, want = a.keep - a.first - a.recent;  // `want` of the `mid` from j0 on
    if (rank == 0) {
        for (int i = tid; i < a.first; i += kSelThreads) out[i] = i;
        for (int i = tid; i < a.recent; i += kSelThreads) out[a.first + want + i] = j0 + mid + i;
    }
    if (want == 0) return;
    if (plan.ctas > 1) cluster_arrive();  // waited for below: the first CTA runs before the others write to it
    uint32_t* keys = GLOBAL ? a.scores + (long long)bh * a.stride : s_keys;  // of block j0 + i
    const uint32_t keys0 = mapa_shared(smem_u32(s_keys), 0);                 // those of the first CTA
    const __nv_bfloat16* bounds = (const __nv_bfloat16*)a.bounds;
    // the row of `bounds` (2 D elements) of block j, ~0u without a page; its entry of the table is loaded beforehand
    auto entry_of = [&](int j) { return a.table[(long long)b * a.max_pages + (int)plan.per_page.div(j)]; };
    auto row_at = [&](int j, int pg) {
        if ((unsigned)pg >= (unsigned)a.num_pages) {
            record_invalid(a.err, kSiteCacheTable, pg);
            return ~0u;
        }
        return ((uint32_t)pg * a.Hkv + kvh) * bpp + (uint32_t)(j - (int)plan.per_page.div(j) * bpp);
    };
    auto row_of = [&](int j) { return row_at(j, entry_of(j)); };
    const int share = ((mid + plan.ctas - 1) / plan.ctas + kBatch - 1) & ~(kBatch - 1), i0 = rank * share, i1 = min(i0 + share, mid);
    const int g8 = lane >> 2, t4 = lane & 3;
    auto entries_of = [&](int g) { return lane < kBatch && g + lane < i1 ? entry_of(j0 + g + lane) : 0; };
    uint32_t big[S], lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
    for (int s = 0; s < S; ++s) big[s] = 0;
    for (int r0 = 0; r0 < a.rows; r0 += kRowTile) {
        const int many = min(kRowTile, a.rows - r0);
        int g = i0 + warp * kBatch;
        int entries = entries_of(g);
        if (r0 > 0) {
            __syncthreads();
            stage(r0, many);
        }
        uint4 w[2][S];  // of blocks g8 and g8 + 8 of the batch
        auto load = [&](int g) {
            const uint32_t rows = lane < kBatch && g + lane < i1 ? row_at(j0 + g + lane, entries) : ~0u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t row = __shfl_sync(0xffffffffu, rows, g8 + 8 * h);
                const uint4* src = reinterpret_cast<const uint4*>(bounds + (size_t)(row != ~0u ? row : 0) * (2 * D)) + t4;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if (RING)
                        copy16(smem_u32(s_ring + (h * S + s) * THREADS), src + s * 4, row != ~0u);
                    else
                        w[h][s] = row != ~0u ? src[s * 4] : make_uint4(0, 0, 0, 0);
                }
            }
            if (RING) asm volatile("cp.async.commit_group;" ::: "memory");
        };
        load(g);
        entries = entries_of(g + kSelWarps * kBatch);
        __syncthreads();
        if (r0 == 0 && plan.ctas > 1) cluster_wait();
        for (; g < i1; g += kSelWarps * kBatch) {
            const int next = g + kSelWarps * kBatch;
            if (RING) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int s = 0; s < S; ++s) w[h][s] = s_ring[(h * S + s) * THREADS];
                if (next < i1) load(next);
                entries = entries_of(next + kSelWarps * kBatch);
            }
            float best[2] = {-INFINITY, -INFINITY};
            for (int n = 0; n * 8 < many; ++n) {
                float c[4][4] = {};
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const uint4 x = s_q[(n * S + s) * 32 + lane];
                    mma_bf16(c[2 * s % 4], w[0][s].x, w[1][s].x, w[0][s].y, w[1][s].y, x.x, x.y);
                    mma_bf16(c[(2 * s + 1) % 4], w[0][s].z, w[1][s].z, w[0][s].w, w[1][s].w, x.z, x.w);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)  // rows 2 t4 + k % 2 of block g8 + 8 (k / 2)
                    if (n * 8 + 2 * t4 + k % 2 < many) best[k / 2] = fmaxf(best[k / 2], (c[0][k] + c[1][k]) + (c[2][k] + c[3][k]));
            }
#pragma unroll
            for (int s = 0; s < S; ++s) {
                big[s] = abs_max2(abs_max2(big[s], w[0][s].x), w[0][s].y);
                big[s] = abs_max2(abs_max2(big[s], w[0][s].z), w[0][s].w);
                big[s] = abs_max2(abs_max2(big[s], w[1][s].x), w[1][s].y);
                big[s] = abs_max2(abs_max2(big[s], w[1][s].z), w[1][s].w);
            }
            if (!RING) {
                if (next < i1) load(next);
                entries = entries_of(next + kSelWarps * kBatch);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                best[h] = fmaxf(best[h], __shfl_xor_sync(0xffffffffu, best[h], 1));
                best[h] = fmaxf(best[h], __shfl_xor_sync(0xffffffffu, best[h], 2));
                const int i = g + g8 + 8 * h;
                if (t4 == 0 && i < i1) {
                    uint32_t key = key32(best[h]);
                    if (GLOBAL) {
                        if (r0 > 0) key = max(keys[i], key);
                        keys[i] = key;
                    } else {
                        st_cluster_u32(keys0 + 4 * i, key);
                    }
                    if (r0 + kRowTile >= a.rows) lo = min(lo, key), hi = max(hi, key);
                }
            }
        }
    }
    // ---- what the cluster found goes to its first CTA
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) big[s] = abs_max2(big[s], __shfl_xor_sync(0xffffffffu, big[s], m));
        if (g8 == 0) atomicMax(&s_big[s * 4 + t4], max(big[s] << 16, big[s] & 0xFFFF0000u));
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        atomicMax(&s_big[CHUNKS], ~lo);
        atomicMax(&s_big[CHUNKS + 1], hi);
    }
    __syncthreads();
    if (rank > 0 && tid < CHUNKS + 2)
        asm volatile("red.shared::cluster.max.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&s_big[tid]), 0)), "r"(s_big[tid]) : "memory");
    if (plan.ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank > 0) return;
    // ---- the first CTA chooses.  A warp has a run of the scores, the lanes in turn.
    const int run = ((mid + kSelWarps - 1) / kSelWarps + 31) & ~31, wi = warp * run, we = min(wi + run, mid);
    auto each = [&](auto f) {  // f(i, key)
        int i = wi + lane;
        for (; i + 96 < we; i += 128) {
            const uint32_t k[4] = {keys[i], keys[i + 32], keys[i + 64], keys[i + 96]};
#pragma unroll
            for (int u = 0; u < 4; ++u) f(i + 32 * u, k[u]);
        }
        for (; i < we; i += 32) f(i, keys[i]);
    };
    int turn = 0;
    // sums over the CTA, the same in every thread; buffers alternate, so one barrier per call is enough
    auto block_sums = [&](int x, int y) {
        x = __reduce_add_sync(0xffffffffu, x);
        y = __reduce_add_sync(0xffffffffu, y);
        turn ^= 1;
        if (lane == 0) s_sum[turn][warp] = make_int2(x, y);
        __syncthreads();
        const int2 v = lane < kSelWarps ? s_sum[turn][lane] : make_int2(0, 0);
        return make_int2(__reduce_add_sync(0xffffffffu, v.x), __reduce_add_sync(0xffffffffu, v.y));
    };
    lo = ~s_big[CHUNKS], hi = s_big[CHUNKS + 1];
    float A = 0.f;  // the largest sum of |q_c| |bound_c| that a row can have; NaN and infinities stay
    if (lane < CHUNKS) A = __uint_as_float(s_sum8[lane]) * __uint_as_float(s_big[lane]);
    for (int w = 16; w >= 1; w >>= 1) A += __shfl_xor_sync(0xffffffffu, A, w);
    const float E = kError * 1.001f * A + 1e-30f;  // A itself is rounded; products may underflow
    // a score stays if its key is above `over`, or from `from` on and picked by the exact scores
    uint32_t from = 0, over = 0xFFFFFFFFu;
    int left = want, near = mid;
    bool open = true;  // some are undecided and not all of them stay
    const bool finite = E < 1e33f;  // every score, and E's parts
    if (finite) {
        // the smallest key that stays, T: the bin that it is in, then itself
        uint32_t T = lo;
        int need = want;  // of those in [lo, hi]
        while (lo < hi) {
            const int shift = max(0, 32 - __clz(hi - lo) - 10);  // at most kBins bins
            each([&](int, uint32_t k) {
                if (k >= lo && k <= hi) atomicAdd(&s_hist[(k - lo) >> shift], 1);
            });
            __syncthreads();
            constexpr int PER = kBins / THREADS;  // bins of a thread, from the top down
            int c[PER], sum = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += c[i] = s_hist[kBins - 1 - (tid * PER + i)];
            int incl = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += up;
            }
            turn ^= 1;
            if (lane == 31) s_sum[turn][warp].x = incl;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PER; ++i) s_hist[kBins - 1 - (tid * PER + i)] = 0;
            int above = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[turn][lane].x : 0);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (above < need && need <= above + c[i]) {
                    s_found[0] = kBins - 1 - (tid * PER + i);
                    s_found[1] = above;
                    s_many = c[i];
                }
                above += c[i];
            }
            __syncthreads();
            const int bin = s_found[0], many = s_many;
            need -= s_found[1];
            lo += (uint32_t)bin << shift;
            hi = min(hi, lo + ((1u << shift) - 1));
            T = lo;
            if (many <= kList && lo < hi) {  // count greater ones within the bin
                __syncthreads();
                if (tid == 0) s_many = 0;
                __syncthreads();
                each([&](int, uint32_t k) {
                    if (k >= lo && k <= hi) s_list[atomicAdd(&s_many, 1)] = k;
                });
                __syncthreads();
                if (tid < many) {
                    const uint32_t k = s_list[tid];
                    int greater = 0, same = 0;
                    for (int i = 0; i < many; ++i) greater += s_list[i] > k, same += s_list[i] == k;
                    if (greater < need && need <= greater + same) s_key = k;
                }
                __syncthreads();
                T = s_key;
                break;
            }
        }
        over = key32(score_of(T) + 2.5f * E);
        from = key32(score_of(T) - 2.5f * E);
        int above = 0, there = 0;
        each([&](int, uint32_t k) {
            above += k > over;
            there += k >= from && k <= over;
        });
        const int2 sums = block_sums(above, there);
        left = want - sums.x;
        near = sums.y;
        open = near > left;
    }
    // ---- exact scores of the undecided, a warp for each, 8 lanes for each row: sums of whole numbers, in units of 2^-61 A
    // (what is lost below them is 2^-58 A at most), or, where something is not finite or tiny, in fp64, which has next
    // to no throughput here (a block of 32 rows took 40 us).  What is decided by them is written over the scores: the largest
    // key or the smallest.
    const bool fixed = finite && A >= 1e-12f;  // no product that counts is subnormal
    auto exact_key = [&](int i) -> uint64_t {
        const uint32_t row = row_of(j0 + i);
        const int part = lane & 7;
        // a product is taken apart in whole multiples of 2^21 / A, 2^43 / A and 2^65 / A (A rounded up to a power of two),
        // each found by adding 1.5 x 2^23, which rounds to whole numbers, and exact to take off
        constexpr float kMagic = 12582912.f;
        const float one = __uint_as_float((uint32_t)(127 + 21 + 126 - (fixed ? (int)(__float_as_uint(A) >> 23) : 127)) << 23);
        const uint4* at = reinterpret_cast<const uint4*>(bounds + (size_t)(row != ~0u ? row : 0) * (2 * D));
        constexpr int C = D / 64;
        uint4 l[C], h[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            l[c] = row != ~0u ? at[c * 8 + part] : make_uint4(0, 0, 0, 0);
            h[c] = row != ~0u ? at[D / 8 + c * 8 + part] : make_uint4(0, 0, 0, 0);
        }
        uint64_t top = 0;
        uint4 next[C];  // the next row
        auto load_row = [&](int r) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                next[c] = reinterpret_cast<const uint4*>(q + (long long)min(r, a.rows - 1) * D)[c * 8 + part];
        };
        load_row(lane >> 3);
#pragma unroll 1
        for (int r = lane >> 3; r < ((a.rows + 3) & ~3); r += 4) {
            uint4 row4[C];
#pragma unroll
            for (int c = 0; c < C; ++c) row4[c] = next[c];
            load_row(r + 4);
            uint64_t key;
            if (fixed) {
                int s0 = 0, s1 = 0, s2 = 0;
                auto add = [&](float qe, float le, float he) {
                    float x = qe * (qe < 0.f ? le : he) * one;  // at most 2^21
                    auto whole = [&](int& s) {
                        const float t = x + kMagic;
                        s += __float_as_int(t) - __float_as_int(kMagic);
                        x = (x - (t - kMagic)) * 4194304.f;
                    };
                    whole(s0);
                    whole(s1);
                    whole(s2);
                };
                auto add2 = [&](uint32_t x, uint32_t l, uint32_t h) {
                    add(__uint_as_float(x << 16), __uint_as_float(l << 16), __uint_as_float(h << 16));
                    add(__uint_as_float(x & 0xFFFF0000u), __uint_as_float(l & 0xFFFF0000u), __uint_as_float(h & 0xFFFF0000u));
                };
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint4 x = row4[c];
                    add2(x.x, l[c].x, h[c].x);
                    add2(x.y, l[c].y, h[c].y);
                    add2(x.z, l[c].z, h[c].z);
                    add2(x.w, l[c].w, h[c].w);
                }
#pragma unroll
                for (int m = 1; m < 8; m <<= 1) {  // |s| <= 128 x 2^22
                    s0 += __shfl_xor_sync(0xffffffffu, s0, m);
                    s1 += __shfl_xor_sync(0xffffffffu, s1, m);
                    s2 += __shfl_xor_sync(0xffffffffu, s2, m);
                }
                // in units of 2^-61 A, which 64 bits hold: the last part rounded to them
                key = (uint64_t)(((long long)s0 << 40) + ((long long)s1 << 18) + ((s2 + 8) >> 4)) ^ (1ull << 63);
            } else {
                key = slow_key(q + (long long)min(r, a.rows - 1) * D, row != ~0u ? reinterpret_cast<const __nv_bfloat16*>(at) : nullptr, D, part);
            }
            top = max(top, key);  // NaN on top
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
        return max(top, __shfl_xor_sync(0xffffffffu, top, 16));
    };
    if (open && near <= kList) {
        __syncthreads();
        if (tid == 0) s_many = 0;
        __syncthreads();
        each([&](int i, uint32_t k) {
            if (k >= from && k <= over) s_list[atomicAdd(&s_many, 1)] = i;
        });
        __syncthreads();
        for (int u = warp; u < near; u += kSelWarps) {
            const uint64_t e = exact_key((int)s_list[u]);
            if (lane == 0) s_exact[u] = e;
        }
        __syncthreads();
        if (tid < near) {
            const uint64_t e = s_exact[tid];
            int before = 0;
            for (int u = 0; u < near; ++u) before += s_exact[u] > e || (s_exact[u] == e && s_list[u] < s_list[tid]);
            keys[s_list[tid]] = before < left ? 0xFFFFFFFFu : 0;
        }
        __syncthreads();
        from = max(from, 1u);
    } else if (open) {
        uint64_t* exact = reinterpret_cast<uint64_t*>(a.exact) + (long long)bh * a.stride;
        auto undecided = [&](int i, uint32_t k) { return i < we && k >= from && k <= over; };
        for (int g = wi; g < we; g += 32) {
            uint32_t todo = __ballot_sync(0xffffffffu, undecided(g + lane, g + lane < we ? keys[g + lane] : 0));
            while (todo) {
                const int l = __ffs(todo) - 1;
                todo &= todo - 1;
                const uint64_t e = exact_key(g + l);
                if (lane == 0) exact[g + l] = e;
            }
        }
        __syncthreads();
        auto each_open = [&](auto f) {
            each([&](int i, uint32_t k) {
                if (k >= from && k <= over) f(exact[i]);
            });
        };
        uint64_t least = 0;  // of the exact keys that stay; of those equal to it the first `equal`
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t cand = least | 1ull << bit;
            int c = 0;
            each_open([&](uint64_t k) { c += k >= cand; });
            if (block_sums(c, 0).x >= left) least = cand;
        }
        int above = 0, same = 0;
        each_open([&](uint64_t k) { above += k > least, same += k == least; });
        const int equal = left - block_sums(above, 0).x;
        same = __reduce_add_sync(0xffffffffu, same);
        turn ^= 1;
        if (lane == 0) s_sum[turn][warp].x = same;
        __syncthreads();
        int ties = __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[turn][lane].x : 0);  // before this warp's
        for (int g = wi; g < we; g += 32) {
            const int i = g + lane;
            const uint32_t k = i < we ? keys[i] : 0;
            const bool u = undecided(i, k);
            const uint64_t e = u ? exact[i] : 0;
            const uint32_t eq = __ballot_sync(0xffffffffu, u && e == least);
            if (u) keys[i] = e > least || (e == least && ties + __popc(eq & ((1u << lane) - 1)) < equal) ? 0xFFFFFFFFu : 0;
            ties += __popc(eq);
        }
        __syncthreads();
        from = max(from, 1u);
    }
    // ---- the places of those that stay, in order: the warps' counts first
    int kept = 0;
    each([&](int, uint32_t k) { kept += k >= from; });
    kept = __reduce_add_sync(0xffffffffu, kept);
    turn ^= 1;
    if (lane == 0) s_sum[turn][warp].x = kept;
    __syncthreads();
    out += a.first + __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[turn][lane].x : 0);
    constexpr int U = 4;
    for (int g = wi; g < we; g += 32 * U) {
        uint32_t in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = g + 32 * u + lane;
            in[u] = __ballot_sync(0xffffffffu, i < we && keys[i] >= from);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (in[u] >> lane & 1) out[__popc(in[u] & ((1u << lane) - 1))] = j0 + g + 32 * u + lane;
            out += __popc(in[u]);
        }
    }
}

template <int THREADS>
constexpr int kSmem = (THREADS == 512 ? 226 : 112) * 1024 - 10 * 1024;  // dynamic, beside the rest

template <int D, bool GLOBAL, int THREADS>
cudaError_t launch_t(const SelectLaunch& a, const SelectPlan& plan, int smem, cudaStream_t s) {
    cudaError_t e = set_smem_limit_once<select_blocks_kernel<D, GLOBAL, THREADS>>(kSmem<THREADS>);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * plan.ctas));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)plan.ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, select_blocks_kernel<D, GLOBAL, THREADS>, a, plan);
}

// Scores in shared memory while they and the rest fit (with 256 threads, twice on an SM), else in the workspace.
template <int D, int THREADS>
cudaError_t launch_s(const SelectLaunch& a, const SelectPlan& plan, long long cap, cudaStream_t s) {
    const int fixed = (THREADS == 256 ? D / 8 * THREADS * 16 : 0) + plan.tiles * D * 32;
    if (a.rows <= kRowTile && cap <= (kSmem<THREADS> - fixed) / 4)
        return launch_t<D, false, THREADS>(a, plan, fixed + (int)cap * 4, s);
    return launch_t<D, true, THREADS>(a, plan, fixed, s);
}

template <int D>
cudaError_t launch_d(const SelectLaunch& a, cudaStream_t s) {
    SelectPlan plan;
    const int bpp = a.page_blocks;
    plan.per_page = FastDiv((uint32_t)bpp);
    // CTAs per (sequence, kv head): more while each has a batch for every warp and all of them fit at once
    const long long bh = (long long)a.B * a.Hkv, cap = (long long)a.max_pages * bpp;
    plan.ctas = 1;
    while (plan.ctas < kSelectCtas && cap > 128ll * plan.ctas && bh * plan.ctas <= a.num_sms) plan.ctas *= 2;
    const bool wide = bh * plan.ctas <= a.num_sms;  // a CTA has an SM to itself
    plan.tiles = (std::min(a.rows, kRowTile) + 7) / 8;
    return wide ? launch_s<D, 512>(a, plan, cap, s) : launch_s<D, 256>(a, plan, cap, s);
}

}  // namespace

cudaError_t launch_select_blocks(const SelectLaunch& a, cudaStream_t s) {
    return a.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace fa
