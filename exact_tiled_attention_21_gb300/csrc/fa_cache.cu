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
#include "fa_e4m3.cuh"
#include "fa_internal.h"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kHalf = 128;  // threads of a block's K half (the V half has as many)

// Largest value over the 128 threads of a half (w: 0 for K, 1 for V), the same in each of them.
__device__ __forceinline__ uint32_t half_max(uint32_t v, uint32_t (&s)[2][4], int w) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) s[w][(threadIdx.x >> 5) & 3] = v;
    __syncthreads();
    return max(max(s[w][0], s[w][1]), max(s[w][2], s[w][3]));
}

// Smallest power of two s >= 2^-126 with amax <= 448 s, from the bits of a bf16 amax: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(uint32_t amax_bf16) {
    const int e = (int)(amax_bf16 >> 7) - 8 + ((amax_bf16 & 0x7F) > 0x60 ? 1 : 0);  // biased exponent of s
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// Magnitude bits of the two finite bf16 of a word (infinities and NaN count as 0: they saturate or stay NaN).
__device__ __forceinline__ uint32_t amax2(uint32_t w) {
    const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
    return max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u);
}

__device__ __forceinline__ uint2 quantise8(uint4 x, float inv, float s, bool pow2) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[4] = {bf_lo(w[2 * i]), bf_hi(w[2 * i]), bf_lo(w[2 * i + 1]), bf_hi(w[2 * i + 1])};
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = pow2 ? f[j] * inv : __fdiv_rn(f[j], s);
        r[i] = e4m3x4(f[0], f[1], f[2], f[3]);
    }
    return make_uint2(r[0], r[1]);
}

// One CTA per (sequence, touched block of sb tokens, kv head); the first 128 threads take K, the others V.
// A thread holds TPT tasks (16 columns of a token: the pieces that a rotation pairs) in registers between the
// block's maximum and the quantisation, so new tokens are read once.  If the scale grows, the block's earlier
// tokens are requantised in place.
template <int D, int TPT, bool INTER>
__global__ void __launch_bounds__(2 * kHalf) cache_append_kernel(const CacheAppendLaunch a, int blocks) {
    __shared__ uint32_t s_max[2][4];
    pdl_launch_dependents();
    pdl_wait();
    constexpr int TPR = D / 16;
    const int h = blockIdx.x % a.Hkv;
    const int blk = (blockIdx.x / a.Hkv) % blocks;
    const int b = blockIdx.x / a.Hkv / blocks;
    const int is_v = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
    const int cap = a.max_pages * a.page;
    int len = a.lens[b], n = a.new_lens ? a.new_lens[b] : a.N;
    if (len < 0 || len > cap || n < 0 || n > a.N || n > cap - len) {
        if (threadIdx.x == 0) record_invalid(a.err, kSiteCacheLen, len);
        len = min(max(len, 0), cap);
        n = min(min(max(n, 0), a.N), cap - len);
    }
    const int first = (len / a.sb + blk) * a.sb;  // the block's first token
    if (first >= len + n) return;
    const int pg = a.table[(long long)b * a.max_pages + first / a.page];
    if ((unsigned)pg >= (unsigned)a.num_pages) {
        if (threadIdx.x == 0) record_invalid(a.err, kSiteCacheTable, pg);
        return;
    }
    const int at = first % a.page;  // token within the page
    const long long head = (long long)pg * a.Hkv + h;
    uint8_t* dst = (is_v ? a.vp : a.kp) + (head * a.page + at) * D;
    float* sc = (is_v ? a.vs : a.ks) + head * (a.page / a.sb) + at / a.sb;
    const int t0 = max(len - first, 0), t1 = min(a.sb, len + n - first);  // new tokens [t0, t1) of the block
    const __nv_bfloat16* src = is_v ? (const __nv_bfloat16*)a.v + b * a.vb + h * a.vh
                                    : (const __nv_bfloat16*)a.k + b * a.kb + h * a.kh;
    const long long sn = is_v ? a.vn : a.kn;

    uint4 x[TPT], y[TPT];
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const int task = tid + i * kHalf, tok = task / TPR, p = task % TPR;
        if (tok < t0 || tok >= t1) continue;
        const int idx = first + tok - len;
        int c0, c1;
        task_columns<INTER>(p, is_v || !a.turns ? 0 : a.rot, c0, c1);
        x[i] = *reinterpret_cast<const uint4*>(src + idx * sn + c0);
        y[i] = *reinterpret_cast<const uint4*>(src + idx * sn + c1);
    }
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const int task = tid + i * kHalf, tok = task / TPR, p = task % TPR;
        if (tok < t0 || tok >= t1) continue;
        if (!is_v && a.turns && p < a.rot / 16) {
            const int idx = first + tok - len;
            const int pos = a.positions ? a.positions[(long long)b * a.N + idx] : len + idx;
            float c[8], s[8];
            task_cos_sin(pos, a.turns + p * 8, a.magnitude, c, s);
            rotate16<INTER>(x[i], y[i], c, s);  // rounded to bf16: the bytes of fa_rope followed by this append
        }
        big = max(big, max(max(amax2(x[i].x), amax2(x[i].y)), max(amax2(x[i].z), amax2(x[i].w))));
        big = max(big, max(max(amax2(y[i].x), amax2(y[i].y)), max(amax2(y[i].z), amax2(y[i].w))));
    }
    const float old = t0 > 0 ? *sc : 0.f;
    const float to = fmaxf(old, scale_for(half_max(big, s_max, is_v)));  // every thread has read the old scale
    const bool pow2 = (__float_as_uint(to) & 0x7FFFFFu) == 0 && to >= 1.17549435e-38f && to <= 1.7e38f;
    const float inv = pow2 ? __uint_as_float((254u << 23) - __float_as_uint(to)) : 0.f;
    if (to != old) {
        for (int i = tid; i < t0 * TPR; i += kHalf) {
            uint4* at16 = reinterpret_cast<uint4*>(dst) + i;
            *at16 = e4m3_rescale16(*at16, old, to);
        }
        if (tid == 0) *sc = to;
    }
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const int task = tid + i * kHalf, tok = task / TPR, p = task % TPR;
        if (tok < t0 || tok >= t1) continue;
        int c0, c1;
        task_columns<INTER>(p, is_v || !a.turns ? 0 : a.rot, c0, c1);
        const uint2 u = quantise8(x[i], inv, to, pow2), w = quantise8(y[i], inv, to, pow2);
        uint8_t* row = dst + tok * D;
        if (c1 == c0 + 8) {
            *reinterpret_cast<uint4*>(row + c0) = make_uint4(u.x, u.y, w.x, w.y);
        } else {
            *reinterpret_cast<uint2*>(row + c0) = u;
            *reinterpret_cast<uint2*>(row + c1) = w;
        }
    }
}

template <int D, int TPT>
cudaError_t launch_append_dt(const CacheAppendLaunch& a, cudaStream_t s) {
    const int blocks = (a.N + a.sb - 2) / a.sb + 1;  // of sb tokens that N tokens can touch
    const long long ctas = (long long)a.B * blocks * a.Hkv;
    if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)ctas), block(2 * kHalf);
    return a.interleaved ? launch_dependent(cache_append_kernel<D, TPT, true>, grid, block, 0, s, a, blocks)
                         : launch_dependent(cache_append_kernel<D, TPT, false>, grid, block, 0, s, a, blocks);
}

template <int D>
cudaError_t launch_append_d(const CacheAppendLaunch& a, cudaStream_t s) {
    const int tasks = a.sb * (D / 16);  // of a block, at most 8 per thread (sb <= 128)
    if (tasks <= kHalf) return launch_append_dt<D, 1>(a, s);
    if (tasks <= 2 * kHalf) return launch_append_dt<D, 2>(a, s);
    if (tasks <= 4 * kHalf) return launch_append_dt<D, 4>(a, s);
    return launch_append_dt<D, 8>(a, s);
}

// ------------------------------------------------------------------ eviction
// Which tokens stay: the last `recent`, and of the others the keep - recent with the largest weights (ties: lowest
// index).  One CTA per (sequence, kv head): a radix selection over the weights' order-preserving integer keys finds
// the smallest key that stays and how many equal ones do; a pass in index order then writes the list.
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;

// Integer whose order is the float's, with -0 = +0 and NaN above everything.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0xFFFFFFFFu;
    if (w == 0.f) w = 0.f;
    const uint32_t u = __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const CacheEvictLaunch a) {
    __shared__ uint32_t s_hist[2048];
    __shared__ uint32_t s_warp[kSelWarps];
    __shared__ uint32_t s_digit, s_left;
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cap = a.max_pages * a.page, ncap = a.new_max_pages * a.page;
    int n = a.lens[b];
    if (n < 0 || n > cap) {
        if (tid == 0) record_invalid(a.err, kSiteCacheLen, n);
        n = min(max(n, 0), cap);
    }
    const int stay = min(n, a.keep);
    if (h == 0 && tid == 0) a.new_lens[b] = stay;
    const float* w = a.weights + (long long)blockIdx.x * cap;
    int* kept = a.kept + (long long)blockIdx.x * ncap;
    float* nw = a.new_weights + (long long)blockIdx.x * ncap;
    for (int j = stay + tid; j < ncap; j += kSelThreads) {
        kept[j] = -1;
        nw[j] = 0.f;
    }
    if (n <= a.keep) {
        for (int j = tid; j < n; j += kSelThreads) {
            kept[j] = j;
            nw[j] = w[j];
        }
        return;
    }
    const int cand = n - a.recent;  // candidates [0, cand): `left` of them stay
    uint32_t left = (uint32_t)(a.keep - a.recent), key = 0, known = 0;  // key's bits under the mask `known` are settled
    if (left > 0) {
        int shift = 21;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < 2048; i += kSelThreads) s_hist[i] = 0;
            __syncthreads();
            for (int j = tid; j < cand; j += kSelThreads) {
                const uint32_t k = order_key(w[j]);
                if ((k & known) == key) atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            // bins from the largest down: thread t holds bins 2047 - 2t and 2046 - 2t
            const uint32_t c0 = s_hist[2047 - 2 * tid], c1 = s_hist[2046 - 2 * tid];
            uint32_t sum = c0 + c1, incl = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += up;
            }
            if (lane == 31) s_warp[warp] = incl;
            __syncthreads();
            uint32_t before = incl - sum;
            for (int i = 0; i < warp; ++i) before += s_warp[i];
            if (before < left && before + sum >= left) {  // exactly one thread
                const bool second = before + c0 < left;
                s_digit = (uint32_t)(2047 - 2 * tid - (second ? 1 : 0));
                s_left = left - before - (second ? c0 : 0);
            }
            __syncthreads();
            key |= s_digit << shift;
            known |= ((1u << bits) - 1) << shift;
            left = s_left;
            shift -= pass == 0 ? 11 : 10;
            __syncthreads();
        }
    } else {
        key = 0xFFFFFFFFu;  // none of the candidates: no equal one is admitted either
    }
    // in index order: keys above `key` stay, and the first `left` equal ones
    uint32_t base = 0, equal_base = 0;
    for (int j0 = 0; j0 < n; j0 += kSelThreads) {
        const int j = j0 + tid;
        float wj = 0.f;
        bool above = false, equal = false;
        if (j < n) {
            wj = w[j];
            const uint32_t k = order_key(wj);
            above = j >= cand || (k > key);
            equal = j < cand && k == key;
        }
        const uint32_t ma = __ballot_sync(0xffffffffu, above), me = __ballot_sync(0xffffffffu, equal);
        __syncthreads();  // the previous round's sums have been read
        if (lane == 0) s_warp[warp] = __popc(ma) | (__popc(me) << 16);
        __syncthreads();
        uint32_t pre = 0, all = 0;
        for (int i = 0; i < kSelWarps; ++i) {
            const uint32_t v = s_warp[i];
            if (i < warp) pre += v;
            all += v;
        }
        const uint32_t below = (1u << lane) - 1;
        const uint32_t ra = base + (pre & 0xFFFFu) + __popc(ma & below);                // kept by key before j
        const uint32_t re = equal_base + (pre >> 16) + __popc(me & below);              // equal ones before j
        if (above || (equal && re < left)) {
            const uint32_t at = ra + min(re, left);
            kept[at] = j;
            nw[at] = wj;
        }
        base += all & 0xFFFFu;
        equal_base += all >> 16;
    }
}

// One CTA per (sequence, kv head, block of sb kept tokens): K by the first 128 threads, V by the others.  The block's
// scale is the largest of its tokens' source scales; tokens that came with that scale are copied byte for byte.
template <int D, int TPT>
__global__ void __launch_bounds__(2 * kHalf) evict_move_kernel(const CacheEvictLaunch a) {
    __shared__ uint32_t s_max[2][4];
    pdl_launch_dependents();
    pdl_wait();
    constexpr int TPR = D / 16;
    const int blocks = (a.keep + a.sb - 1) / a.sb;
    const int blk = blockIdx.x % blocks;
    const long long bh = blockIdx.x / blocks;
    const int b = (int)(bh / a.Hkv), h = (int)(bh % a.Hkv);
    const int is_v = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
    const int cap = a.max_pages * a.page, ncap = a.new_max_pages * a.page;
    const int stay = min(min(max(a.lens[b], 0), cap), a.keep);
    const int first = blk * a.sb, count = min(a.sb, stay - first);
    if (count <= 0) return;
    const int npg = a.new_table[(long long)b * a.new_max_pages + first / a.page];
    if ((unsigned)npg >= (unsigned)a.num_pages) {
        if (threadIdx.x == 0) record_invalid(a.err, kSiteCacheTable, npg);
        return;
    }
    const int at = first % a.page, bpp = a.page / a.sb;
    const long long nhead = (long long)npg * a.Hkv + h;
    uint8_t* dst = (is_v ? a.vp : a.kp) + (nhead * a.page + at) * D;
    const uint8_t* pool = is_v ? a.vp : a.kp;
    const float* scales = is_v ? a.vs : a.ks;
    const int* kept = a.kept + bh * ncap + first;
    uint4 x[TPT];
    float sc[TPT];
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const int task = tid + i * kHalf, tok = task / TPR;
        x[i] = make_uint4(0, 0, 0, 0);
        sc[i] = 0.f;
        if (tok >= count) continue;
        const int j = kept[tok];
        const int pg = a.table[(long long)b * a.max_pages + j / a.page];
        if ((unsigned)pg >= (unsigned)a.num_pages) {
            record_invalid(a.err, kSiteCacheTable, pg);  // reads as zeros
            continue;
        }
        const int o = j % a.page;
        const long long head = (long long)pg * a.Hkv + h;
        sc[i] = scales[head * bpp + o / a.sb];
        x[i] = *reinterpret_cast<const uint4*>(pool + (head * a.page + o) * D + (task % TPR) * 16);
        big = max(big, __float_as_uint(fabsf(sc[i])));  // scales are positive: their bits order as they do
    }
    const float to = __uint_as_float(half_max(big, s_max, is_v));
    if (tid == 0) (is_v ? a.vs : a.ks)[nhead * bpp + at / a.sb] = to;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const int task = tid + i * kHalf;
        if (task / TPR >= count) continue;
        reinterpret_cast<uint4*>(dst)[task] = sc[i] == to ? x[i] : e4m3_rescale16(x[i], sc[i], to);
    }
}

template <int D>
cudaError_t launch_move(const CacheEvictLaunch& a, cudaStream_t s) {
    const long long ctas = (long long)a.B * a.Hkv * ((a.keep + a.sb - 1) / a.sb);
    if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)ctas), block(2 * kHalf);
    const int tasks = a.sb * (D / 16);
    if (tasks <= kHalf) return launch_dependent(evict_move_kernel<D, 1>, grid, block, 0, s, a);
    if (tasks <= 2 * kHalf) return launch_dependent(evict_move_kernel<D, 2>, grid, block, 0, s, a);
    if (tasks <= 4 * kHalf) return launch_dependent(evict_move_kernel<D, 4>, grid, block, 0, s, a);
    return launch_dependent(evict_move_kernel<D, 8>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendLaunch& a, cudaStream_t s) {
    return a.d == 128 ? launch_append_d<128>(a, s) : launch_append_d<64>(a, s);
}

cudaError_t launch_cache_evict(const CacheEvictLaunch& a, cudaStream_t s) {
    cudaError_t e = launch_dependent(evict_select_kernel, dim3((unsigned)a.B * a.Hkv), dim3(kSelThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    return a.d == 128 ? launch_move<128>(a, s) : launch_move<64>(a, s);
}

}  // namespace fa
