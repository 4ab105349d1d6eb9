// The attention of fa_decode_rows.cuh as a kernel of its own, and the merge of its parts and of a shared prefix's.
#include "fa_decode_rows.cuh"

namespace fa {
namespace {

template <int D, int ROWS, bool DRAFTS, bool LIST>
__global__ void __launch_bounds__(kThreads, Cfg<D, ROWS>::CTAS) decode_rows_kernel(const Params a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RowsShared<ROWS> sh;
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0) check_lengths(a.lens, a.B, a.max_pages * (int)a.page.d, LIST ? 0 : *a.shared, a.err);
    decode_rows<D, ROWS, DRAFTS, LIST, false>(a, smem, sh, threadIdx.x, blockIdx.x, a.workers, 0);
}

// ------------------------------------------------------------------ merge
// LSE = M + log2 sum 2^(lse_s - M), O = sum 2^(lse_s - M) o_s / sum over a row's parts.  D / 4 threads per row and group;
// SPLIT: one row per block, its parts dealt to the groups, else a row per group.  A row without keys gets O = 0, LSE = -inf.
template <int D, int ROWS, bool LIST, bool SPLIT, int THREADS>
__global__ void __launch_bounds__(THREADS) merge_rows_kernel(const Params a) {
    constexpr int LANES = D / 4, GROUPS = THREADS / LANES, AHEAD = 4;
    __shared__ float4 s_o[SPLIT ? GROUPS : 1][LANES];
    __shared__ float2 s_ms[SPLIT ? GROUPS : 1];
    pdl_wait();
    const int tid = threadIdx.x, grp = tid / LANES, col = tid % LANES;
    const long long all = (long long)a.B * a.Hkv * a.rows, row = SPLIT ? blockIdx.x : (long long)blockIdx.x * GROUPS + grp;
    if (row >= all) return;
    const int bh = (int)a.per_row.div((uint32_t)row), r = (int)row - bh * a.rows, b = (int)a.heads.div(bh),
              kvh = bh - b * a.Hkv, rt = r / ROWS;
    const Parts x = find_parts<LIST>(a, b, kvh, rt, r);
    if (x.done) return;
    const int n = x.n + x.pn, prow = LIST ? 0 : (b * a.rows + r) % a.pre_rows;
    auto lse_at = [&](int s) {
        return s < x.n ? a.part_lse[(x.slot + s) * ROWS + (r - rt * ROWS)]
                       : a.pre_lse[(x.pslot + s - x.n) * a.pre_rows + prow];
    };
    auto o_at = [&](int s) {
        return reinterpret_cast<const float4*>(s < x.n ? a.part_o + ((x.slot + s) * ROWS + (r - rt * ROWS)) * D
                                                       : a.pre_o + ((x.pslot + s - x.n) * a.pre_rows + prow) * D)[col];
    };
    float m = -INFINITY, sum = 0.f;  // running maximum and sum of this group's parts
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int STRIDE = SPLIT ? GROUPS : 1;
    for (int s0 = SPLIT ? grp : 0; s0 < n; s0 += AHEAD * STRIDE) {
        float w[AHEAD];
        float4 v[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int s = s0 + i * STRIDE;
            w[i] = s < n ? lse_at(s) : -INFINITY;
            v[i] = s < n ? o_at(s) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) top = fmaxf(top, w[i]);
        const float base = top == -INFINITY ? 0.f : top, f = ex2(m - base);
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
        sum *= f;
        m = top;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float e = ex2(w[i] - base);
            sum += e;
            if (e != 0.f) {  // a part without keys is zero, whatever is in its place; NaN stays
                o.x = fmaf(e, v[i].x, o.x);
                o.y = fmaf(e, v[i].y, o.y);
                o.z = fmaf(e, v[i].z, o.z);
                o.w = fmaf(e, v[i].w, o.w);
            }
        }
    }
    if constexpr (SPLIT) {
        s_o[grp][col] = o;
        if (col == 0) s_ms[grp] = make_float2(m, sum);
        __syncthreads();
        if (grp > 0) return;
        float top = m;
#pragma unroll
        for (int i = 1; i < GROUPS; ++i) top = fmaxf(top, s_ms[i].x);
        const float base = top == -INFINITY ? 0.f : top;
        sum = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const float f = ex2(s_ms[i].x - base);
            sum += s_ms[i].y * f;
            if (f != 0.f) {
                const float4 y = s_o[i][col];
                o.x = fmaf(f, y.x, o.x);
                o.y = fmaf(f, y.y, o.y);
                o.z = fmaf(f, y.z, o.z);
                o.w = fmaf(f, y.w, o.w);
            }
        }
        m = top;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(a.o + row * D + col * 4) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (a.lse && col == 0) a.lse[row] = sum == 0.f ? -INFINITY : (m + lg2(sum)) * kLn2;
}

template <int D, int ROWS, bool LIST>
cudaError_t launch_merge(const DecodeRowsLaunch& a, const Params& p, cudaStream_t s) {
    const long long rows = (long long)a.B * a.Hkv * p.rows;
    // Rows alone in a block where there are few of them: their parts are read by more threads, 8 groups of them where a row has
    // many parts (288 rows of about 76: 24.2 us in 8 groups, 27.2 in 4; 1024 rows of about 19: 23.8 and 22.8; four rows to a
    // block 47 and 25.9; 4096 rows of about 9: 99.7, 95.2 and 93.8 with four to a block, the whole call each).  Where one kernel
    // has the prefix and own tokens, about half of its CTAs have the prefix.
    const long long most = LIST ? (long long)a.keep * a.block : (long long)a.max_pages * a.page,
                    ctas = LIST ? p.workers : a.joint ? p.workers / 2 : a.merge_only ? a.pre_workers / 2 : a.pre_workers,
                    parts = std::min(ctas / (LIST ? (long long)a.B * a.Hkv * p.row_tiles : (long long)a.Hkv * p.pre_tiles),
                                     most / Cfg<D, ROWS>::STEP);
    if (rows <= (parts >= 4 ? 16ll : 4ll) * a.num_sms)
        return parts >= 16 ? launch_dependent(merge_rows_kernel<D, ROWS, LIST, true, 256>, dim3((unsigned)rows), dim3(256), 0, s, p)
                           : launch_dependent(merge_rows_kernel<D, ROWS, LIST, true, 128>, dim3((unsigned)rows), dim3(128), 0, s, p);
    constexpr int PER = 128 / (D / 4);
    return launch_dependent(merge_rows_kernel<D, ROWS, LIST, false, 128>, dim3((unsigned)((rows + PER - 1) / PER)), dim3(128), 0,
                            s, p);
}

template <int D, int ROWS>
cudaError_t launch_clusters(const DecodeRowsLaunch& a, const Params& p, int ctas, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D, ROWS>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)p.cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return a.Nq > 1 ? cudaLaunchKernelEx(&cfg, decode_rows_kernel<D, ROWS, true, true>, p)
                    : cudaLaunchKernelEx(&cfg, decode_rows_kernel<D, ROWS, false, true>, p);
}

template <int D, int ROWS, bool LIST>
cudaError_t launch_l(const DecodeRowsLaunch& a, cudaStream_t s) {
    using C = Cfg<D, ROWS>;
    cudaError_t e = a.Nq > 1 ? set_smem_limit_once<decode_rows_kernel<D, ROWS, true, LIST>>(C::SMEM)
                             : set_smem_limit_once<decode_rows_kernel<D, ROWS, false, LIST>>(C::SMEM);
    if (e != cudaSuccess) return e;
    Params p = rows_params<D, ROWS>(a);
    if (a.merge_only) return launch_merge<D, ROWS, LIST>(a, p, s);
    // no more CTAs than steps at full lengths
    const long long most = LIST ? std::min((long long)a.keep * a.block, (long long)a.max_pages * a.page + a.block)
                                : (long long)a.max_pages * a.page;
    const int slots = std::min(C::CTAS * a.num_sms, kRowsMostWorkers);  // CTAs that run at once
    const long long items = (long long)a.B * a.Hkv * p.row_tiles;
    if (LIST && items <= slots) {
        p.cluster = 1;
        const long long steps = (most + C::STEP - 1) / C::STEP;  // of an item
        while (p.cluster < kMostCluster && items * p.cluster * 2 <= slots && steps > p.cluster) p.cluster *= 2;
        // unless a few items leave most SMs idle: the second kernel costs about three steps (8 items of 64 steps: 11.5 us in
        // clusters, 9.5 in shares; 32 of 10: 10.2 and 12.2; 256 of 16, alone: 25.4 and 28.5)
        if ((steps + p.cluster - 1) / p.cluster <= (steps * items + slots - 1) / slots + 3)
            return launch_clusters<D, ROWS>(a, p, (int)(items * p.cluster), s);
        p.cluster = 0;
    }
    p.workers = (int)std::min<long long>(slots,
                                         ((long long)a.B + p.tiles) * a.Hkv * p.row_tiles * ((most + C::STEP - 1) / C::STEP));
    if (a.joint) p.pre_workers = p.workers;
    e = launch_dependent(a.Nq > 1 ? decode_rows_kernel<D, ROWS, true, LIST> : decode_rows_kernel<D, ROWS, false, LIST>,
                         dim3(p.workers), dim3(kThreads), C::SMEM, s, p);
    return e != cudaSuccess ? e : launch_merge<D, ROWS, LIST>(a, p, s);
}

template <int D, int ROWS>
cudaError_t launch_r(const DecodeRowsLaunch& a, cudaStream_t s) {
    return a.list ? launch_l<D, ROWS, true>(a, s) : launch_l<D, ROWS, false>(a, s);
}

}  // namespace

cudaError_t launch_decode_rows(const DecodeRowsLaunch& a, cudaStream_t s) {
    const int tile = a.merge_only ? 8 : rows_tile(a.joint ? a.joint : a.Hq / a.Hkv * a.Nq);
    if (a.d == 128) return tile == 8 ? launch_r<128, 8>(a, s) : tile == 16 ? launch_r<128, 16>(a, s) : launch_r<128, 32>(a, s);
    return tile == 8 ? launch_r<64, 8>(a, s) : tile == 16 ? launch_r<64, 16>(a, s) : launch_r<64, 32>(a, s);
}

}  // namespace fa
