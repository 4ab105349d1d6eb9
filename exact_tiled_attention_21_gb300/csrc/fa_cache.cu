// The paged 8-bit cache: writing new tokens into it, and moving the tokens that
// an eviction keeps.
//
// Layout: e4m3 bytes [num_pages, Hkv, page, d] for K and for V, fp32 scales
// [num_pages, Hkv, page / sb], one per block of sb consecutive tokens of a page.
// An element stands for its e4m3 value times its block's scale.  The append
// writes powers of two: dividing by one is exact and rescaling a block moves
// only exponents, so a token's bytes do not depend on which later tokens raised
// its block's scale (unless they become subnormal); e4m3's relative step
// is the same at every scale, so nothing is lost against amax / 448 either.
#include <algorithm>

#include "fa_e4m3.cuh"
#include "fa_internal.h"
#include "fa_rope.cuh"

namespace fa {
namespace {


// Largest value over the 32 W threads of a block's half (w: 0 for K, 1 for V), the same in each of them.
template <int W>
__device__ __forceinline__ uint32_t half_max(uint32_t v, uint32_t (&s)[2][W], int w) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) s[w][(threadIdx.x >> 5) % W] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) v = max(v, s[w][i]);
    return v;
}

// The same over the threads of a block of sb tokens, where a half holds several and every token has TPR threads: `token`
// is the thread's and `first` its block's first one.
template <int W, int TPR>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t (&s)[2][32 * W / TPR], int w, int token, int first, int sb) {
#pragma unroll
    for (int d = 1; d < TPR; d <<= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
    s[w][token] = v;
    __syncthreads();
    for (int i = first; i < min(first + sb, 32 * W / TPR); ++i) v = max(v, s[w][i]);
    return v;
}

// Smallest power of two s >= 2^-126 with amax <= 448 s, from the bits of a bf16 amax: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(uint32_t amax_bf16) {
    const int e = (int)(amax_bf16 >> 7) - 8 + ((amax_bf16 & 0x7F) > 0x60 ? 1 : 0);  // biased exponent of s
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// Largest magnitudes of the two halves of bf16 pairs; NaN wins.
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
    return r;
}
__device__ __forceinline__ uint32_t abs_max(uint4 x, uint4 y) {
    const uint32_t a = abs_max2(abs_max2(abs_max2(x.x, x.y), abs_max2(x.z, x.w)), abs_max2(abs_max2(y.x, y.y), abs_max2(y.z, y.w)));
    uint32_t m = max(a & 0x7FFFu, (a >> 16) & 0x7FFFu);
    if (m >= 0x7F80u) {  // infinities and NaN: the largest finite one (they saturate, or stay NaN)
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        m = 0;
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            const uint32_t v = (w[i / 2] >> (i % 2 * 16)) & 0x7FFFu;
            if (v < 0x7F80u) m = max(m, v);
        }
    }
    return m;
}

// Eight bf16 as e4m3 bytes of their values divided by s; pow2: by its exact inverse.
__device__ __forceinline__ uint2 quantise8(uint4 x, float inv, float s, bool pow2) {
    if (pow2) {  // as bf16 pairs: exact but for what underflows, which rounds to zero either way
        const uint32_t two = __byte_perm(__float_as_uint(inv), 0, 0x3232);
        asm("mul.bf16x2 %0, %0, %1;" : "+r"(x.x) : "r"(two));
        asm("mul.bf16x2 %0, %0, %1;" : "+r"(x.y) : "r"(two));
        asm("mul.bf16x2 %0, %0, %1;" : "+r"(x.z) : "r"(two));
        asm("mul.bf16x2 %0, %0, %1;" : "+r"(x.w) : "r"(two));
    }
    float f[8] = {bf_lo(x.x), bf_hi(x.x), bf_lo(x.y), bf_hi(x.y), bf_lo(x.z), bf_hi(x.z), bf_lo(x.w), bf_hi(x.w)};
    if (!pow2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], s);
    }
    return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
}

// One CTA per (sequence, touched block of sb tokens, run of kv heads); the first HALF threads take K, the others V.  Of
// blocks too small for 128 threads a CTA takes several (one with blocks of 4 tokens, 17 sequences of 5624 tokens, 1 head:
// 101 us against 44).  The block's cosines and sines are made once, in shared memory, and serve every head of the run: with
// a pair of them per head and element the sines alone were half of the instructions.  A thread holds TPT tasks (16
// columns of a token: the pieces that a rotation pairs) in registers between the block's maximum and the quantisation,
// so new tokens are read once, the next head's while this one's are worked on.  If the scale grows, the block's earlier
// tokens are requantised in place.  Reads two bytes per element and writes one; bound by instructions, about 240 per warp
// and 512 elements (54% of the ALU pipe): 8 ragged prompts of up to 2048 tokens, 8 heads, d = 128, calls back to back 21.8
// us (3.5 TB/s; 22.6 with the products by the inverse scale in fp32); one token of each of 32 sequences 6.1 us, the latency
// of a launch and four dependent loads.
struct AppendPlan {
    int unit, units, heads, groups;  // blocks per CTA, and runs of them that N tokens can touch; the same of kv heads
    FastDiv page, sb;
};

// Threads of an SM: as many as their registers leave without spills (8 sequences of 2048 tokens in blocks of 32: 28.7 us
// with 768, 33.1 with 1024).
template <int TPT>
constexpr int kAppendThreads = TPT > 2 ? 512 : TPT == 2 ? 768 : 1024;

// SEV: the CTA has several blocks (of HALF threads or fewer in all, one task each).
template <int D, int HALF, int TPT, bool SEV, bool INTER>
__global__ void __launch_bounds__(2 * HALF, kAppendThreads<TPT> / (2 * HALF))
    cache_append_kernel(const CacheAppendLaunch a, const AppendPlan plan) {
    extern __shared__ __align__(16) float2 s_turn[];  // [token][pair of pairs j < 4][task][2]
    constexpr int TPR = D / 16;
    __shared__ uint32_t s_max[2][2][HALF / 32], s_block[2][2][SEV ? HALF / TPR : 1];
    pdl_launch_dependents();
    pdl_wait();
    const int group = blockIdx.x % plan.groups;
    const int unit = (blockIdx.x / plan.groups) % plan.units;
    const int b = blockIdx.x / plan.groups / plan.units;
    const int is_v = threadIdx.x / HALF, tid = threadIdx.x % HALF;
    const int cap = a.max_pages * a.page;
    int len = a.lens[b], n = a.new_lens ? a.new_lens[b] : a.N;
    if (len < 0 || len > cap || n < 0 || n > a.N || n > cap - len) {
        if (threadIdx.x == 0) record_invalid(a.err, kSiteCacheLen, len);
        len = min(max(len, 0), cap);
        n = min(min(max(n, 0), a.N), cap - len);
    }
    const int first = ((int)plan.sb.div(len) + unit * plan.unit) * a.sb;  // the CTA's first token
    if (n == 0 || first >= len + n) return;  // without new tokens the block that len lies in is not touched either
    const int t0 = max(len - first, 0), t1 = min(plan.unit * a.sb, len + n - first);  // its new tokens [t0, t1)
    // the thread's block: its first token (of the CTA's), the earlier tokens in it, its page and place in it
    const int own = SEV ? (int)plan.sb.div(tid / TPR) * a.sb : 0, begin = first + own;
    const int earlier = max(t0 - own, 0);
    bool mine = !SEV || own < t1;
    const int lpage = mine ? (int)plan.page.div(begin) : 0, at = mine ? begin - lpage * a.page : 0;
    const int pg = a.table[(long long)b * a.max_pages + lpage];
    if (mine && (unsigned)pg >= (unsigned)a.num_pages) {
        if (threadIdx.x == own * TPR) record_invalid(a.err, kSiteCacheTable, pg);
        if (!SEV) return;
        mine = false;
    }
    const int turned = a.turns ? a.rot / 16 : 0;  // tasks of a row that rotate
    if (turned) {
        const int q = threadIdx.x % 64;  // one pair for each of up to 64 threads, four tokens at a time
        if (q < turned * 8) {
            const uint64_t turns = a.turns[q];
            for (int tok = t0 + threadIdx.x / 64; tok < t1; tok += 2 * HALF / 64) {
                const int pos = a.positions ? a.positions[(long long)b * a.N + first + tok - len] : first + tok;
                float2 cs;
                turn_cos_sin(pos, turns, a.magnitude, cs.x, cs.y);
                s_turn[((tok * 4 + q % 8 / 2) * turned + q / 8) * 2 + q % 2] = cs;
            }
        }
        __syncthreads();
    }
    // what a task needs in every head: its pieces' columns and places
    const int nb = (int)plan.sb.div(a.page), h0 = group * plan.heads, h1 = min(h0 + plan.heads, a.Hkv);
    const long long sn = is_v ? a.vn : a.kn, sh = is_v ? a.vh : a.kh;
    const __nv_bfloat16* src[TPT];
    int out[TPT], apart[TPT];  // offset of the first piece in the block, and from it to the second; apart = 0: no token
    const float2* cs[TPT];
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const int task = tid + i * HALF, tok = task / TPR, p = task % TPR;
        int c0, c1;
        task_columns<INTER>(p, is_v ? 0 : turned * 16, c0, c1);
        apart[i] = (!SEV || mine) && tok >= t0 && tok < t1 ? c1 - c0 : 0;
        out[i] = (tok - own) * D + c0;
        src[i] = (is_v ? (const __nv_bfloat16*)a.v + b * a.vb : (const __nv_bfloat16*)a.k + b * a.kb) +
                 (first + tok - len) * sn + h0 * sh + c0;
        cs[i] = !is_v && p < turned ? s_turn + (tok * 4 * turned + p) * 2 : nullptr;
    }
    uint8_t* dst = (is_v ? a.vp : a.kp) + (((long long)pg * a.Hkv + h0) * a.page + at) * D;
    float* sc = (is_v ? a.vs : a.ks) + ((long long)pg * a.Hkv + h0) * nb + plan.sb.div(at);
    uint4 nx[TPT], ny[TPT];  // the next head's, loaded while this one's are worked on
    float nold;
    auto load = [&](const float* scale) {
        nold = (!SEV || mine) && earlier > 0 ? *scale : 0.f;
#pragma unroll
        for (int i = 0; i < TPT; ++i)
            if (apart[i]) {
                nx[i] = *reinterpret_cast<const uint4*>(src[i]);
                ny[i] = *reinterpret_cast<const uint4*>(src[i] + apart[i]);
                src[i] += sh;
            }
    };
    load(sc);
    for (int h = h0; h < h1; ++h, dst += (long long)a.page * D, sc += nb) {
        uint4 x[TPT], y[TPT];
        const float old = nold;
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < TPT; ++i) x[i] = nx[i], y[i] = ny[i];
        if (h + 1 < h1) load(sc + nb);
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            if (!apart[i]) continue;
            if (cs[i]) {
                float c[8], s[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 v = *reinterpret_cast<const float4*>(cs[i] + j * turned * 2);
                    c[2 * j] = v.x, s[2 * j] = v.y, c[2 * j + 1] = v.z, s[2 * j + 1] = v.w;
                }
                rotate16<INTER>(x[i], y[i], c, s);  // rounded to bf16: the bytes of fa_rope followed by this append
            }
            big = max(big, abs_max(x[i], y[i]));
        }
        if constexpr (SEV)
            big = block_max<HALF / 32, TPR>(big, s_block[h & 1], is_v, tid / TPR, own, a.sb);
        else
            big = half_max(big, s_max[h & 1], is_v);
        const float to = fmaxf(old, scale_for(big));     // all threads have read the old scale
        const bool pow2 = is_pow2(to) && to <= 1.7e38f;  // 1 / to is normal
        const float inv = pow2 ? __uint_as_float((254u << 23) - __float_as_uint(to)) : 0.f;
        if ((!SEV || mine) && to != old) {
            for (int i = tid - own * TPR; i < earlier * TPR; i += HALF) {
                uint4* at16 = reinterpret_cast<uint4*>(dst) + i;
                *at16 = e4m3_rescale16(*at16, old, to);
            }
            if (tid == own * TPR) *sc = to;
        }
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            if (!apart[i]) continue;
            const uint2 u = quantise8(x[i], inv, to, pow2), w = quantise8(y[i], inv, to, pow2);
            if (apart[i] == 8) {
                *reinterpret_cast<uint4*>(dst + out[i]) = make_uint4(u.x, u.y, w.x, w.y);
            } else {
                *reinterpret_cast<uint2*>(dst + out[i]) = u;
                *reinterpret_cast<uint2*>(dst + out[i] + apart[i]) = w;
            }
        }
    }
}

template <int D, int HALF, int TPT, bool SEV, bool INTER>
cudaError_t launch_append_dti(const CacheAppendLaunch& a, cudaStream_t s) {
    AppendPlan plan;
    const int blocks = (a.N + a.sb - 2) / a.sb + 1;  // that N tokens can touch
    plan.unit = SEV ? std::min(HALF / (a.sb * (D / 16)), blocks) : 1;
    plan.units = (blocks + plan.unit - 1) / plan.unit;
    plan.page = FastDiv((uint32_t)a.page);
    plan.sb = FastDiv((uint32_t)a.sb);
    // kv heads per CTA, which share the sines: the fewest waves of resident CTAs times the work of one, whose start
    // counts for one and a half heads (8 sequences of 2048 tokens, 8 heads, d = 128: with blocks of 32 tokens 1 head 37.3
    // us, 2 28.8, 4 28.1, 8 30.3; blocks of 128 tokens 51.3 for 2 heads, 39.0 for 8; 32 single tokens 6.2 for 1, 8.9 for 8)
    const long long cells = (long long)a.B * plan.units, slots = (long long)kAppendThreads<TPT> / (2 * HALF) * a.num_sms;
    long long best = -1;
    for (int h = 8; h >= 1; h /= 2) {
        const long long waves = (cells * ((a.Hkv + h - 1) / h) + slots - 1) / slots, cost = waves * (2 * h + 3);
        if (best < 0 || cost < best) best = cost, plan.heads = h;
    }
    plan.groups = (a.Hkv + plan.heads - 1) / plan.heads;
    const long long ctas = cells * plan.groups;
    const int smem = a.turns ? plan.unit * a.sb * (a.rot / 2) * 8 : 0;  // at most 64 KB
    cudaError_t e = set_smem_limit_once<cache_append_kernel<D, HALF, TPT, SEV, INTER>>(64 * 1024);
    if (e != cudaSuccess) return e;
    return launch_dependent(cache_append_kernel<D, HALF, TPT, SEV, INTER>, dim3((unsigned)ctas), dim3(2 * HALF), (size_t)smem, s, a,
                            plan);
}

template <int D, int HALF, int TPT, bool SEV>
cudaError_t launch_append_dt(const CacheAppendLaunch& a, cudaStream_t s) {
    return a.interleaved ? launch_append_dti<D, HALF, TPT, SEV, true>(a, s)
                         : launch_append_dti<D, HALF, TPT, SEV, false>(a, s);
}

template <int D>
cudaError_t launch_append_d(const CacheAppendLaunch& a, cudaStream_t s) {
    const int tasks = a.sb * (D / 16);  // of a block (sb <= 128)
    if (tasks <= 64) return launch_append_dt<D, 128, 1, true>(a, s);
    if (tasks <= 128) return launch_append_dt<D, 128, 1, false>(a, s);
    if (tasks <= 256) return launch_append_dt<D, 128, 2, false>(a, s);
    if (tasks <= 512) return launch_append_dt<D, 128, 4, false>(a, s);
    return launch_append_dt<D, 256, 4, false>(a, s);
}

// ------------------------------------------------------------------ eviction
// Which tokens stay: the last `recent`, and of the others the keep - recent with the largest weights (ties: lowest
// index).  A cluster of 1 to 8 CTAs per (sequence, kv head), each with a run of the tokens, whose order-preserving
// integer keys stay in its registers: up to four histograms of 8 bits, summed over the cluster's shared memories, find
// the smallest key that stays and how many equal ones do, and how many of either the CTAs before this one have; a count
// per warp then gives every kept token its place in index order.  The weights are read once.  A round after which the
// digit's keys all stay is the last (for weights without many equal ones the third: 36.2 -> 35.1 us for 1024 of 4096
// tokens, 32 sequences, 8 heads).  Bound by latency: rounds of shared-memory atomics and of exchange between the CTAs, 14
// us for one sequence of 64k tokens, whose eviction takes 24 us (28 with three histograms of 11, 11 and 10 bits, which move
// six times the bins).
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kSelBins = 256, kSelCtas = 8;

// Integer whose order is the float's, with -0 = +0 and NaN above everything.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0xFFFFFFFFu;
    if (w == 0.f) w = 0.f;
    const uint32_t u = __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// PER: keys of a thread in registers (0: any number; they are read again in each pass).
template <int PER>
__global__ void __launch_bounds__(kSelThreads, PER > 8 ? 1 : 2) evict_select_kernel(const CacheEvictLaunch a, int ctas) {
    __shared__ uint32_t s_hist[4][kSelBins];
    __shared__ uint2 s_warp[kSelBins / 32];
    __shared__ uint32_t s_above[kSelWarps], s_equal[kSelWarps], s_digit, s_left, s_prior[2];
    pdl_launch_dependents();
    pdl_wait();
    const int rank = blockIdx.x % ctas;
    const long long bh = blockIdx.x / ctas;
    const int b = (int)(bh / a.Hkv);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cap = a.max_pages * a.page, ncap = a.new_max_pages * a.page;
    int n = a.lens[b];
    if (n < 0 || n > cap) {
        if (tid == 0 && rank == 0) record_invalid(a.err, kSiteCacheLen, n);
        n = min(max(n, 0), cap);
    }
    const int stay = min(n, a.keep);
    if (bh % a.Hkv == 0 && rank == 0 && tid == 0) a.new_lens[b] = stay;
    const float* w = a.weights + bh * cap;
    int* kept = a.kept + bh * ncap;
    float* nw = a.new_weights + bh * ncap;
    for (int j = stay + rank * kSelThreads + tid; j < ncap; j += ctas * kSelThreads) {
        kept[j] = -1;
        nw[j] = 0.f;
    }
    if (n <= a.keep) {  // the whole cluster alike
        for (int j = rank * kSelThreads + tid; j < n; j += ctas * kSelThreads) {
            kept[j] = j;
            nw[j] = w[j];
        }
        return;
    }
    // this CTA's run of tokens, cut into a run for each warp; a warp takes 32 consecutive tokens at a time
    const int per_warp = ((n + ctas * kSelWarps - 1) / (ctas * kSelWarps) + 31) / 32 * 32;
    const int first = (rank * kSelWarps + warp) * per_warp + lane, rounds = per_warp / 32;
    const int cand = n - a.recent;  // candidates [0, cand): `left` of them stay
    // of this thread's tokens first + 32 i: candidates are those with i < ic, recent ones those with ic <= i < in
    const int ic = min(max(cand - first + 31, 0) / 32, rounds), in = min(max(n - first + 31, 0) / 32, rounds);
    float held[PER ? PER : 1] = {};  // loaded all at once, from clamped places
    uint32_t keys[PER ? PER : 1] = {};
    if constexpr (PER > 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) held[i] = w[min(first + i * 32, n - 1)];
    }
    for (int i = tid; i < 4 * kSelBins; i += kSelThreads) s_hist[0][i] = 0;
    if (tid < 2) s_prior[tid] = 0;
    __syncthreads();
    if constexpr (PER > 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) keys[i] = order_key(held[i]);
    }
    auto key_of = [&](int i) { return PER ? keys[PER ? i : 0] : order_key(w[first + i * 32]); };
    uint32_t left = (uint32_t)(a.keep - a.recent), key = 0, known = 0;  // key's bits under the mask `known` are settled
    if (left > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            uint32_t* hist = s_hist[pass];
            const int shift = 24 - 8 * pass;
#pragma unroll
            for (int i = 0; i < (PER ? PER : rounds); ++i)
                if (i < ic) {
                    const uint32_t k = key_of(i);
                    if ((k & known) == key) atomicAdd(&hist[(k >> shift) & (kSelBins - 1)], 1u);
                }
            if (ctas > 1)
                cluster_sync();
            else
                __syncthreads();
            // bins from the largest down: thread t holds bin 255 - t, of the cluster and of the CTAs before this one
            const uint32_t* bin = hist + kSelBins - 1 - tid;
            uint32_t c = 0, ours = 0, incl = 0, incl_ours = 0;
            if (tid < kSelBins) {
                if (ctas > 1) {
                    uint32_t v[kSelCtas];
#pragma unroll
                    for (int r = 0; r < kSelCtas; ++r) v[r] = r < ctas ? ld_cluster_u32(bin, r) : 0;
#pragma unroll
                    for (int r = 0; r < kSelCtas; ++r) {
                        c += v[r];
                        if (r < rank) ours += v[r];
                    }
                } else {
                    c = *bin;
                }
                incl = c, incl_ours = ours;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
                    const uint32_t up_ours = __shfl_up_sync(0xffffffffu, incl_ours, d);
                    if (lane >= d) incl += up, incl_ours += up_ours;
                }
                if (lane == 31) s_warp[warp] = make_uint2(incl, incl_ours);
            }
            __syncthreads();
            if (tid < kSelBins) {
                const uint2 x = lane < warp ? s_warp[lane] : make_uint2(0, 0);
                const uint32_t seen = __reduce_add_sync(0xffffffffu, x.x) + incl - c;
                const uint32_t seen_ours = __reduce_add_sync(0xffffffffu, x.y) + incl_ours - ours;
                if (seen < left && seen + c >= left) {  // exactly one thread
                    const uint32_t digit = kSelBins - 1 - tid, all = seen + c == left && (key | digit << shift) > 0;
                    s_digit = digit;
                    s_left = all ? 0 : left - seen;
                    s_prior[0] += seen_ours + (all ? ours : 0);
                    s_prior[1] = ours;  // equal so far: the last pass's stays
                }
            }
            __syncthreads();
            key |= s_digit << shift;
            known |= (kSelBins - 1) << shift;
            left = s_left;
            if (left == 0) {  // every key with these bits stays: the lower bits need not be known
                --key;
                break;
            }
        }
    } else {
        key = 0xFFFFFFFFu;  // none of the candidates: no equal one is admitted either
    }
    if (ctas > 1) cluster_arrive();  // this CTA has read the others' histograms
    // in index order: keys above `key` and the recent tokens stay, and the first `left` equal ones
    uint32_t above = 0, equal = 0;
#pragma unroll
    for (int i = 0; i < (PER ? PER : rounds); ++i)
        if (i < ic) {
            const uint32_t k = key_of(i);
            above += k > key;
            equal += k == key;
        }
    above += in - ic;
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    // counts before this warp: of the CTA's other warps, and of the cluster's CTAs before this one
    if (lane == 0) s_above[warp] = above, s_equal[warp] = equal;
    __syncthreads();
    uint32_t ba = __reduce_add_sync(0xffffffffu, lane < warp ? s_above[lane] : 0) + s_prior[0];
    uint32_t be = __reduce_add_sync(0xffffffffu, lane < warp ? s_equal[lane] : 0) + s_prior[1];
    ba += (uint32_t)max(min(rank * kSelWarps * per_warp, n) - cand, 0);  // recent tokens among them
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < (PER ? PER : rounds); ++i)
        if (i < rounds) {
            const int j = first + i * 32;
            const uint32_t k = i < ic ? key_of(i) : 0;
            const bool up = i < ic ? k > key : i < in, eq = i < ic && k == key;
            const uint32_t ma = __ballot_sync(0xffffffffu, up), me = equal ? __ballot_sync(0xffffffffu, eq) : 0;
            const uint32_t ra = ba + __popc(ma & below), re = be + __popc(me & below);  // before j
            if (up || (eq && re < left)) {
                const uint32_t at = ra + min(re, left);
                kept[at] = j;
                nw[at] = PER ? held[PER ? i : 0] : w[j];
            }
            ba += __popc(ma);
            be += __popc(me);
        }
    if (ctas > 1) cluster_wait();  // the others have read this CTA's
}

// Moves the kept tokens, a block of sb of them per turn of a CTA (of small blocks several: with blocks of 4 tokens, 7
// sequences of 4681 kept tokens, 8 heads, one takes 103 us against 50): K by the first HALF threads, V by the others.  A
// block's scale is the largest of its tokens' source scales; tokens that came with that scale are copied byte for byte.
// Reading a token takes three loads that depend on each other (its index, its page, its row), so the CTAs are resident
// ones that run over the blocks with the index two blocks ahead and the page one block ahead of the row.  Bound by HBM:
// 134 MB for 1024 of up to 4096 tokens of 32 sequences of 8 heads in about 24 of the eviction's 33.9 us, 5.6 TB/s.
// Threads of an SM, by the pieces that one holds (the eviction of 32 sequences of 4096 tokens, 8 heads, d = 128: blocks
// of 64 tokens 45.1 us with 512, 38.9 with 768, 36.8 with 1024, 41.7 with 1280; blocks of 16 49.3 with 1024, 43.2 with
// 1536, 43.0 with 2048; 4 sequences of 16k tokens, blocks of 32: 29.1 with 768, 27.8 with 1024, 26.7 with 1536).
template <int TPT, bool SEV>
constexpr int kMoveThreads = SEV ? 1536 : TPT == 1 ? 2048 : TPT == 2 ? 1536 : 1024;

struct MovePlan {
    int unit, units;          // tokens per turn, and turns per (sequence, kv head)
    int step_bh, step_units;  // the grid's size as (sequence, kv head)s and turns
    int bhs;
    FastDiv page, sb, heads;
};

template <int D, int HALF, int TPT, bool SEV>
__global__ void __launch_bounds__(2 * HALF, kMoveThreads<TPT, SEV> / (2 * HALF))
    evict_move_kernel(const CacheEvictLaunch a, const MovePlan plan) {
    constexpr int TPR = D / 16;
    __shared__ uint32_t s_max[2][2][HALF / 32], s_block[2][2][SEV ? HALF / TPR : 1];
    pdl_launch_dependents();
    pdl_wait();
    const int is_v = threadIdx.x / HALF, tid = threadIdx.x % HALF;
    const int ncap = a.new_max_pages * a.page, bpp = (int)plan.sb.div(a.page);
    uint8_t* pool = is_v ? a.vp : a.kp;
    float* scales = is_v ? a.vs : a.ks;
    const int own = SEV ? (int)plan.sb.div(tid / TPR) * a.sb : 0;  // first token of the thread's block in the turn
    const bool leads = tid == own * TPR && own < plan.unit;             // writes the block's scale
    struct Item {
        int bh, first;  // first token (its place among the kept)
    };
    auto advance = [&](Item& it) {
        it.bh += plan.step_bh;
        const int left = plan.units * plan.unit - it.first, step = plan.step_units * plan.unit;
        it.first = step < left ? it.first + step : step - left;
        if (step >= left) ++it.bh;
    };
    // stage 1: the source indices of an item's tokens (-1: none)
    auto load_kept = [&](const Item& it, int (&kept)[TPT]) {
        const int* list = a.kept + (long long)it.bh * ncap + it.first;
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int tok = (tid + i * HALF) / TPR;
            kept[i] = it.bh < plan.bhs && tok < plan.unit && it.first + tok < ncap ? list[tok] : -1;
        }
    };
    // stage 2: their pages, and the page that the thread's block goes to
    auto load_pages = [&](const Item& it, const int (&kept)[TPT], int (&page)[TPT], int& to) {
        const int b = it.bh < plan.bhs ? (int)plan.heads.div(it.bh) : 0;
        const int* trow = a.table + (long long)b * a.max_pages;
#pragma unroll
        for (int i = 0; i < TPT; ++i) page[i] = kept[i] >= 0 ? trow[plan.page.div(kept[i])] : 0;
        to = a.new_table[(long long)b * a.new_max_pages + plan.page.div(SEV ? min(it.first + own, ncap - 1) : it.first)];
    };
    int kept[TPT], page[TPT], kept1[TPT], to_page;
    Item item{(int)(blockIdx.x / plan.units), (int)(blockIdx.x % plan.units) * plan.unit}, next = item;
    load_kept(item, kept);
    advance(next);
    load_kept(next, kept1);
    load_pages(item, kept, page, to_page);
    int turn = 0;
    for (; item.bh < plan.bhs; turn ^= 1) {
        const int h = item.bh - (int)plan.heads.div(item.bh) * a.Hkv;
        uint4 x[TPT];
        float sc[TPT];
        uint32_t big = 0;  // bits of the largest scale (positive: they order as they do) + 1; 0: no token
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            x[i] = make_uint4(0, 0, 0, 0);
            sc[i] = 0.f;
            if (kept[i] < 0) continue;
            if ((unsigned)page[i] >= (unsigned)a.num_pages) {
                record_invalid(a.err, kSiteCacheTable, page[i]);  // reads as zeros
                continue;
            }
            const uint32_t o = kept[i] - plan.page.div(kept[i]) * a.page;
            const uint32_t head = (uint32_t)page[i] * a.Hkv + h;  // rows are counted in 32 bits
            sc[i] = scales[head * bpp + plan.sb.div(o)];
            x[i] = *reinterpret_cast<const uint4*>(pool + (size_t)(head * a.page + o) * D + (tid + i * HALF) % TPR * 16);
        }
        // the stages of the blocks behind this one
        int kept2[TPT], page1[TPT], to_page1;
        Item after = next;
        advance(after);
        load_kept(after, kept2);
        load_pages(next, kept1, page1, to_page1);
#pragma unroll
        for (int i = 0; i < TPT; ++i)
            if (kept[i] >= 0) big = max(big, (__float_as_uint(sc[i]) & 0x7FFFFFFFu) + 1);
        if constexpr (SEV)
            big = block_max<HALF / 32, TPR>(big, s_block[turn], is_v, tid / TPR, own, a.sb);
        else
            big = half_max(big, s_max[turn], is_v);
        if (big) {
            const float to = __uint_as_float(big - 1);
            if ((unsigned)to_page < (unsigned)a.num_pages) {
                const uint32_t to_first = item.first + own, at = to_first - plan.page.div(to_first) * a.page;
                const uint32_t head = (uint32_t)to_page * a.Hkv + h;
                uint4* dst = reinterpret_cast<uint4*>(pool + (size_t)(head * a.page + at) * D);
                if (leads) scales[head * bpp + plan.sb.div(at)] = to;
#pragma unroll
                for (int i = 0; i < TPT; ++i)
                    if (kept[i] >= 0) dst[tid - own * TPR + i * HALF] = sc[i] == to ? x[i] : e4m3_rescale16(x[i], sc[i], to);
            } else if (leads) {
                record_invalid(a.err, kSiteCacheTable, to_page);
            }
        }
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            kept[i] = kept1[i];
            kept1[i] = kept2[i];
            page[i] = page1[i];
        }
        to_page = to_page1;
        item = next;
        next = after;
    }
}

template <int D, int HALF, int TPT, bool SEV>
cudaError_t launch_move_t(const CacheEvictLaunch& a, cudaStream_t s) {
    MovePlan plan;
    plan.unit = a.sb * (SEV ? HALF / (a.sb * (D / 16)) : 1);
    plan.units = (a.keep + plan.unit - 1) / plan.unit;
    plan.bhs = a.B * a.Hkv;
    plan.page = FastDiv((uint32_t)a.page);
    plan.sb = FastDiv((uint32_t)a.sb);
    plan.heads = FastDiv((uint32_t)a.Hkv);
    const long long items = (long long)plan.bhs * plan.units, most = (long long)kMoveThreads<TPT, SEV> / (2 * HALF) * a.num_sms;
    const int grid = (int)(items < most ? items : most);
    plan.step_bh = grid / plan.units;
    plan.step_units = grid % plan.units;
    return launch_dependent(evict_move_kernel<D, HALF, TPT, SEV>, dim3(grid), dim3(2 * HALF), 0, s, a, plan);
}

template <int D>
cudaError_t launch_move(const CacheEvictLaunch& a, cudaStream_t s) {
    const int tasks = a.sb * (D / 16);
    if (tasks <= 64) return launch_move_t<D, 128, 1, true>(a, s);
    if (tasks <= 128) return launch_move_t<D, 128, 1, false>(a, s);
    if (tasks <= 256) return launch_move_t<D, 128, 2, false>(a, s);
    if (tasks <= 512) return launch_move_t<D, 128, 4, false>(a, s);
    return launch_move_t<D, 256, 4, false>(a, s);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendLaunch& a, cudaStream_t s) {
    return a.d == 128 ? launch_append_d<128>(a, s) : launch_append_d<64>(a, s);
}

cudaError_t launch_cache_evict(const CacheEvictLaunch& a, cudaStream_t s) {
    // CTAs per (sequence, kv head): more while that still leaves each 2048 tokens and all of them fit at once (one
    // sequence of 64k tokens, 8 heads, with the move: 1 CTA 208 us, 2 117, 4 28.7, 8 27.5), and while a CTA's registers do
    // not hold its keys (20 sequences of 64k tokens, 8 heads: 1 CTA 236 us, 4 93; 8, with 16 keys per thread, 162)
    const long long bh = (long long)a.B * a.Hkv, cap = (long long)a.max_pages * a.page;
    int ctas = 1;
    while (ctas < kSelCtas &&
           (cap > 32ll * kSelThreads * ctas || (cap >= 4096ll * ctas && bh * ctas * 2 <= a.num_sms)))
        ctas *= 2;
    const long long per = (cap + (long long)ctas * kSelThreads - 1) / ((long long)ctas * kSelThreads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(bh * ctas));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // keys in registers: 8 per thread leave two CTAs per SM (32 sequences of 4096 tokens, 8 heads: 37.8 us; 32 registers
    // 49.4, none 46.5), 32 save a long sequence the reads of later rounds (64k tokens: 27.5 us; none 50.3)
    cudaError_t e = per <= 8    ? cudaLaunchKernelEx(&cfg, evict_select_kernel<8>, a, ctas)
                    : per <= 32 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<32>, a, ctas)
                                : cudaLaunchKernelEx(&cfg, evict_select_kernel<0>, a, ctas);
    if (e != cudaSuccess) return e;
    return a.d == 128 ? launch_move<128>(a, s) : launch_move<64>(a, s);
}

}  // namespace fa
