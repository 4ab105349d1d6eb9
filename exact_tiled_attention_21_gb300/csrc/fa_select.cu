// Selection of the blocks of a paged cache that a query is likely to attend to.
//
// From the bounds that the append keeps of every block (the smallest and the
// largest key element of each column), a row q cannot score more with any key of
// block j than
//     u_j = sum_c max(q_c, 0) max_jc + min(q_c, 0) min_jc,
// and a block's score is the largest u_j of the kv head's query rows.  The first
// blocks, the most recent ones and, of the others, those of largest score stay.
//
// The choice is that of exact scores.  They are summed in fp32: the products of
// bf16 numbers are exact, and at most 9 roundings of 2^-24 follow, each of at most
// A = |q|_1 max |bound|, so a score is within E = 2^-19.9 A.  Blocks further than
// 2 E from the smallest score that stays are decided; if the others do not all
// stay, theirs are summed again in fp64 (whose products and, but for elements 2^30
// apart, sums are exact), and equal ones go by index.
//
// 4 d bytes per block and 4 d flops per block and row: bound by HBM where contexts
// are long, by latency otherwise.  One cluster of up to 8 CTAs per (sequence, kv
// head) shares the scores, through the workspace; its first CTA chooses.
#include <algorithm>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kRowTile = 32;   // query rows in shared memory at once
constexpr int kBatch = 8;      // 16-byte loads in flight per lane
constexpr float kError = 1e-6f;  // E / A: 2^-19.9

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums over W lanes of NV values per lane: lane l (of W) gets those of values l NV / W + k in v[k], k < NV / W.
template <int W, int NV>
__device__ __forceinline__ void lane_sums(float (&v)[NV], int lane) {
#pragma unroll
    for (int m = W / 2, n = NV / 2; m >= 1; m >>= 1, n >>= 1) {
        const bool hi = lane & m;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = hi ? v[i] : v[i + n], keep = hi ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
}

// Integers whose order is the numbers', -0 = +0; of a double also NaN, above everything.
__device__ __forceinline__ uint32_t key32(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key64(double x) {
    if (x != x) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : u | (1ull << 63);
}

// Sum over the CTA, the same in every thread.  Buffers alternate by `turn`, so one barrier per call is enough.
__device__ __forceinline__ int block_sum(int v, int (&s)[2][kSelWarps], int& turn) {
    v = __reduce_add_sync(0xffffffffu, v);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < kSelWarps ? s[turn][threadIdx.x & 31] : 0);
}

struct SelectPlan {
    int ctas;            // of a cluster
    FastDiv per_page;    // blocks of a page
};

// PER: scores that a thread of the choosing CTA holds in registers (0: any number, read again in each pass).
template <int D, int PER>
__global__ void __launch_bounds__(kSelThreads, 1) select_blocks_kernel(const SelectLaunch a, const SelectPlan plan) {
    constexpr int LANES = D / 4, APART = 32 / LANES;  // lanes of a block's bounds; blocks of a warp's load
    constexpr int GROUP = kBatch * APART;             // blocks of a warp's batch
    __shared__ float4 s_q[kRowTile][2][LANES];        // min(q, 0) and max(q, 0): first, then second four of a lane's columns
    __shared__ int s_count[2][kSelWarps];
    __shared__ uint32_t s_big[kSelWarps];
    __shared__ float s_norm[kSelWarps];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % plan.ctas;
    const int bh = blockIdx.x / plan.ctas, b = bh / a.Hkv, kvh = bh - b * a.Hkv;
    const int bpp = (int)plan.per_page.d, cap = a.max_pages * bpp * a.block;
    int len = a.lens[b];
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
    const int j0 = a.first, j1 = n - a.recent, want = a.keep - a.first - a.recent;  // choose `want` of [j0, j1)
    float* scores = a.scores + (long long)bh * a.stride;
    const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + (long long)bh * a.rows * D;
    const __nv_bfloat16* bounds = (const __nv_bfloat16*)a.bounds;
    // the row of `bounds` (2 D elements) of block j, ~0u without a page
    auto row_of = [&](int j) {
        const int lpage = (int)plan.per_page.div(j), pg = a.table[(long long)b * a.max_pages + lpage];
        if ((unsigned)pg >= (unsigned)a.num_pages) {
            record_invalid(a.err, kSiteCacheTable, pg);
            return ~0u;
        }
        return ((uint32_t)pg * a.Hkv + kvh) * bpp + (uint32_t)(j - lpage * bpp);
    };
    float norm = 0.f;   // largest |q|_1 of this warp's rows
    uint32_t big = 0;   // bits of the largest |bound|; infinities and NaN on top
    const int share = (j1 - j0 + plan.ctas - 1) / plan.ctas;
    const int s0 = j0 + rank * share, s1 = min(s0 + share, j1);
    for (int r0 = 0; want > 0 && r0 < a.rows; r0 += kRowTile) {
        const int many = min(kRowTile, a.rows - r0), padded = (many + 3) & ~3;
        if (r0 > 0) __syncthreads();
        for (int r = warp; r < padded; r += kSelWarps) {
            float sum = 0.f;
            for (int c = lane; c < D / 4; c += 32) {  // four columns
                const uint2 w = r < many ? reinterpret_cast<const uint2*>(q + (long long)(r0 + r) * D)[c] : make_uint2(0, 0);
                const float4 x = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                             __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
                // NaN stays in both parts
                auto neg = [](float v) { return v > 0.f ? 0.f : v; };
                auto pos = [](float v) { return v < 0.f ? 0.f : v; };
                s_q[r][c & 1][c >> 1] = make_float4(neg(x.x), neg(x.y), neg(x.z), neg(x.w));
                s_q[r][c & 1][LANES / 2 + (c >> 1)] = make_float4(pos(x.x), pos(x.y), pos(x.z), pos(x.w));
                sum += (fabsf(x.x) + fabsf(x.y)) + (fabsf(x.z) + fabsf(x.w));
            }
            for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            if (!(sum <= norm)) norm = sum;  // NaN stays
        }
        __syncthreads();
        for (int g0 = s0 + warp * GROUP; g0 < s1; g0 += kSelWarps * GROUP) {
            const uint32_t mine = lane < GROUP && g0 + lane < s1 ? row_of(g0 + lane) : ~0u;
            uint4 w[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t row = __shfl_sync(0xffffffffu, mine, i * APART + lane / LANES);
                w[i] = row != ~0u ? *reinterpret_cast<const uint4*>(bounds + (size_t)row * (2 * D) + lane % LANES * 8)
                                  : make_uint4(0, 0, 0, 0);
            }
            float2 x[kBatch][4];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x[i][c] = make_float2(__uint_as_float(u[c] << 16), __uint_as_float(u[c] & 0xFFFF0000u));
                    big = max(big, max(u[c] << 16 & 0x7FFFFFFFu, u[c] & 0x7FFF0000u));
                }
            }
            float best[APART];  // lane l (of LANES): block l APART / 4 ... of the batch (see lane_sums)
#pragma unroll
            for (int k = 0; k < APART; ++k) best[k] = -INFINITY;
            for (int r = 0; r < padded; r += 4) {
                float v[kBatch * 4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 qa = s_q[r + k][0][lane % LANES], qb = s_q[r + k][1][lane % LANES];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        float2 s = ffma2(x[i][0], make_float2(qa.x, qa.y), make_float2(0.f, 0.f));
                        s = ffma2(x[i][1], make_float2(qa.z, qa.w), s);
                        s = ffma2(x[i][2], make_float2(qb.x, qb.y), s);
                        s = ffma2(x[i][3], make_float2(qb.z, qb.w), s);
                        v[i * 4 + k] = s.x + s.y;
                    }
                }
                lane_sums<LANES>(v, lane);  // value l APART + k is load (l APART + k) / 4, row (l APART + k) % 4
#pragma unroll
                for (int k = 0; k < APART; ++k)
                    if (r + (lane * APART + k) % 4 < many) best[k] = fmaxf(best[k], v[k]);
            }
            float top = best[0];
#pragma unroll
            for (int k = 1; k < APART; ++k) top = fmaxf(top, best[k]);
#pragma unroll
            for (int m = 1; m < 4 / APART; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
            const int j = g0 + lane % LANES * APART / 4 * APART + lane / LANES;
            if (lane % (4 / APART) == 0 && j < s1) scores[j] = r0 > 0 ? fmaxf(scores[j], top) : top;
        }
    }
    // ---- what the cluster found goes to its first CTA
    big = __reduce_max_sync(0xffffffffu, big);
    if (lane == 0) s_big[warp] = big, s_norm[warp] = norm;
    __syncthreads();
    big = __reduce_max_sync(0xffffffffu, lane < kSelWarps ? s_big[lane] : 0);
    if (tid == 0) a.big[bh * kSelectCtas + rank] = big;
    if (plan.ctas > 1)
        cluster_barrier();
    else
        __syncthreads();
    if (rank > 0) return;
    // ---- the first CTA: thread t holds V consecutive scores
    const int V = (j1 - j0 + kSelThreads - 1) / kSelThreads, jt = j0 + tid * V, jn = min(V, max(0, j1 - jt));
    uint32_t key[PER ? PER : 1];
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = i < jn && want > 0 ? key32(scores[jt + i]) : 0;
    auto each = [&](auto f) {  // f(block, key of its score)
        if constexpr (PER > 0) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i < jn) f(jt + i, key[i]);
        } else {
            for (int i = 0; i < jn; ++i) f(jt + i, key32(scores[jt + i]));
        }
    };
    int turn = 0;
    // a block stays if its key is above `over`, or from `from` on and picked by the exact scores
    uint32_t from = 0, over = 0xFFFFFFFFu;
    uint64_t exact_from = 0;  // of the undecided: exact keys above it stay, and the first `equal` that are equal to it
    int equal = INT_MAX;
    uint64_t* exact = reinterpret_cast<uint64_t*>(a.exact) + (long long)bh * a.stride;
    if (want > 0) {
        float A = s_norm[0];
        for (int w = 1; w < kSelWarps; ++w)
            if (!(s_norm[w] <= A)) A = s_norm[w];
        uint32_t top = 0;
        for (int r = 0; r < plan.ctas; ++r) top = max(top, a.big[bh * kSelectCtas + r]);
        const float E = kError * 1.01f * (A * __uint_as_float(top)) + 1e-30f;  // A itself is rounded; products may underflow
        bool open = true;  // some are undecided and not all of them stay
        int left = want;   // of the undecided
        if (E < 1e38f) {   // every score is finite
            // the smallest key that stays, bit by bit
            uint32_t T = 0;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t cand = T | 1u << bit;
                int c = 0;
                each([&](int, uint32_t k) { c += k >= cand; });
                c = block_sum(c, s_count, turn);
                if (c >= want) T = cand;
            }
            const float t = __uint_as_float((T & 0x80000000u) ? T ^ 0x80000000u : ~T);
            over = key32(t + 2.5f * E);
            from = key32(t - 2.5f * E);
            int above = 0, near = 0;
            each([&](int, uint32_t k) {
                above += k > over;
                near += k >= from && k <= over;
            });
            above = block_sum(above, s_count, turn);
            near = block_sum(near, s_count, turn);
            left = want - above;
            open = near > left;
        }
        if (open) {
            // exact scores of the undecided, a warp for each
            for (int g = j0 + warp * 32; g < j1; g += kSelThreads) {
                const uint32_t k = g + lane < j1 ? key32(scores[g + lane]) : 0;
                uint32_t todo = __ballot_sync(0xffffffffu, g + lane < j1 && k >= from && k <= over);
                const uint32_t mine = todo >> lane & 1 ? row_of(g + lane) : ~0u;
                while (todo) {
                    const int l = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const uint32_t row = __shfl_sync(0xffffffffu, mine, l);
                    double best = -INFINITY;
                    for (int r = 0; r < a.rows; ++r) {
                        double sum = 0.0;
                        for (int c = lane; c < D; c += 32) {
                            const double qc = (double)__bfloat162float(q[(long long)r * D + c]);
                            const __nv_bfloat16* at = bounds + (size_t)row * (2 * D) + c;
                            const double lo = row != ~0u ? (double)__bfloat162float(at[0]) : 0.0;
                            const double hi = row != ~0u ? (double)__bfloat162float(at[D]) : 0.0;
                            sum += (qc > 0.0 ? 0.0 : qc) * lo + (qc < 0.0 ? 0.0 : qc) * hi;
                        }
                        for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                        if (!(sum <= best)) best = best != best ? best : sum;  // NaN stays
                    }
                    if (lane == 0) exact[g + l] = key64(best);
                }
            }
            __syncthreads();
            auto each_open = [&](auto f) {
                each([&](int j, uint32_t k) {
                    if (k >= from && k <= over) f(exact[j]);
                });
            };
            for (int bit = 63; bit >= 0; --bit) {
                const uint64_t cand = exact_from | 1ull << bit;
                int c = 0;
                each_open([&](uint64_t k) { c += k >= cand; });
                if (block_sum(c, s_count, turn) >= left) exact_from = cand;
            }
            int c = 0;
            each_open([&](uint64_t k) { c += k > exact_from; });
            equal = left - block_sum(c, s_count, turn);
        }
    }
    const bool by_exact = equal != INT_MAX;
    // equal ones before this thread's, then the places of those that stay
    auto before = [&](int mine) {  // exclusive sum over the threads
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
        turn ^= 1;
        if (lane == 31) s_count[turn][warp] = incl;
        __syncthreads();
        return incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? s_count[turn][lane] : 0);
    };
    int ties = 0;
    if (by_exact) {
        int c = 0;
        each([&](int j, uint32_t k) { c += k >= from && k <= over && exact[j] == exact_from; });
        ties = before(c);
    }
    auto stay = [&](auto f) {
        if (want == 0) return;
        int t = ties;
        each([&](int j, uint32_t k) {
            bool in = k > over;
            if (k >= from && k <= over) {
                if (!by_exact) {
                    in = true;
                } else {
                    const uint64_t e = exact[j];
                    in = e > exact_from || (e == exact_from && t < equal);
                    t += e == exact_from;
                }
            }
            if (in) f(j);
        });
    };
    int kept = 0;
    stay([&](int) { ++kept; });
    int at = a.first + before(kept);
    stay([&](int j) { out[at++] = j; });
    for (int i = tid; i < a.first; i += kSelThreads) out[i] = i;
    for (int i = tid; i < a.recent; i += kSelThreads) out[a.first + want + i] = j1 + i;
}

template <int D>
cudaError_t launch_d(const SelectLaunch& a, cudaStream_t s) {
    SelectPlan plan;
    const int bpp = a.page_blocks;
    plan.per_page = FastDiv((uint32_t)bpp);
    // CTAs per (sequence, kv head): more while each has a batch for every warp and all of them fit at once
    const long long bh = (long long)a.B * a.Hkv, cap = (long long)a.max_pages * bpp;
    plan.ctas = 1;
    while (plan.ctas < kSelectCtas && cap > 128ll * plan.ctas && bh * plan.ctas * 2 <= 2 * a.num_sms) plan.ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(bh * plan.ctas));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)plan.ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const long long per = (cap + kSelThreads - 1) / kSelThreads;
    return per <= 1   ? cudaLaunchKernelEx(&cfg, select_blocks_kernel<D, 1>, a, plan)
           : per <= 4 ? cudaLaunchKernelEx(&cfg, select_blocks_kernel<D, 4>, a, plan)
           : per <= 16 ? cudaLaunchKernelEx(&cfg, select_blocks_kernel<D, 16>, a, plan)
                      : cudaLaunchKernelEx(&cfg, select_blocks_kernel<D, 0>, a, plan);
}

}  // namespace

cudaError_t launch_select_blocks(const SelectLaunch& a, cudaStream_t s) {
    return a.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace fa
