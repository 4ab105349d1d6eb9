// The C ABI declared in include/fa.h: argument validation, TMA tensor-map
// encoding, the per-device error word, and the launches.  No allocation, no
// fallback: every call either launches the GPU kernels or returns an error.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <mutex>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {
namespace {

__device__ DevError g_dev_error;  // one per device (per context)

constexpr int kMaxDevices = 64;
std::atomic<uint64_t> g_timeout_ns{2000000000ull};
std::mutex g_mu;
DevError* g_err_addr[kMaxDevices] = {};
int g_num_sms[kMaxDevices] = {};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Per-device state, looked up with the current device active.
int device_state(DevError** err, int* num_sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_err_addr[dev]) {
        void* a = nullptr;
        if (cudaGetSymbolAddress(&a, g_dev_error) != cudaSuccess || !a) return FA_ERR_CUDA;
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
            return FA_ERR_CUDA;
        g_err_addr[dev] = static_cast<DevError*>(a);
        g_num_sms[dev] = sms;
    }
    if (err) *err = g_err_addr[dev];
    if (num_sms) *num_sms = g_num_sms[dev];
    return FA_OK;
}

int encoder(PFN_cuTensorMapEncodeTiled_v12000* fn) {
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_encode) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !f)
            return FA_ERR_CUDA;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    *fn = g_encode;
    return FA_OK;
}

// 3-D map over a contiguous (BH, N, d) bf16 tensor: dims (d, N, BH), box
// (64, 128, 1), 128-byte swizzle (matches the MMA shared-memory descriptors).
int make_map(CUtensorMap* m, const void* base, int BH, int N, int d, unsigned box_rows = 128) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    int st = encoder(&enc);
    if (st != FA_OK) return st;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)N * d * 2};
    cuuint32_t box[3] = {64, box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
                     es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// Tiled map of any rank (bf16, 128-byte swizzle, zero fill out of range).
// strides: bytes of dims 1..rank-1.
int make_map_nd(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                const cuuint32_t* box, CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    int st = encoder(&enc);
    if (st != FA_OK) return st;
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    CUresult r = enc(m, dtype, rank, const_cast<void*>(base), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// Page sizes the tensor-core paged decode takes: whole 8-row swizzle atoms per page.  It loads
// a page in boxes of gcd(page, 128) rows (at least 8), which tile both the page and a 128-key
// stage.
bool paged_mma_ok(int d, int page) { return (d == 64 || d == 128) && page % 8 == 0; }

// Rows of one TMA box of a page: gcd(page, 128) for a multiple of 8.
int page_box_rows(int page) { return std::min(page & -page, 128); }

// Shared shape checks.  Sizes must keep every element index below 2^31 per
// tensor row block and the total within 64-bit byte offsets.
int check_shape(int B, int H, int Nq, int Nk, int d) {
    if (B < 1 || H < 1 || Nq < 1 || Nk < 1) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    const long long BH = (long long)B * H;
    if (BH > (1ll << 24)) return FA_ERR_UNSUPPORTED;  // work-tile indices stay in int
    if ((long long)Nq * BH > (1ll << 36) || (long long)Nk * BH > (1ll << 36)) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

bool scale_ok(float s) { return std::isfinite(s) && s > 0.f; }

// The backward keeps dQ in TMEM (Q-tile-parallel pass), so its only scratch
// is D = rowsum(dO o O): one fp32 per query row.
size_t bwd_ws_bytes(int B, int H, int Nq, int d) {
    (void)d;
    const size_t rows = (size_t)B * H * Nq;
    return (rows * 4 + 255) & ~(size_t)255;
}

int decode_auto_splits(int Nk) {
    // chunks of at least 256 keys, at most 16 chunks
    int s = (Nk + 255) / 256;
    return s < 1 ? 1 : (s > 16 ? 16 : s);
}

int g_dec_blocks[kMaxDevices][2] = {};  // resident split-kernel CTAs per SM, by device and d (64, 128)

// Automatic split count of the contiguous decode on CUDA cores.  One CTA per (b, h, split) keeps a
// fixed number of loads in flight, so a launch costs about waves * (per-CTA time): waves =
// ceil(B*H*splits / resident CTAs), per-CTA time = the split's key pieces plus a fixed cost of
// about one piece (q load, reductions, the partial write), in keys.  Among 1 .. decode_auto_splits(Nk)
// splits it takes the cheapest, the fewest on a tie (fewer partials to merge).  A split count
// that spills a few CTAs into a second wave costs a whole wave: at B=8, H=32, Nk=4000, d=128 (7
// CTAs per SM, 1064 resident) 4 splits read 0.83 of HBM and 6 splits 0.68.
int decode_wave_splits(int B, int H, int Nk, int d, int* splits) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
    int num_sms = 0;
    int st = device_state(nullptr, &num_sms);
    if (st != FA_OK) return st;
    int per_sm = 0;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        int& c = g_dec_blocks[dev][d == 128 ? 1 : 0];
        if (!c) {
            int b = 0;
            if (decode_split_blocks_per_sm(d, &b) != cudaSuccess || b < 1) return FA_ERR_CUDA;
            c = b;
        }
        per_sm = c;
    }
    const long long resident = (long long)num_sms * per_sm, bh = (long long)B * H;
    const long long piece = d == 64 ? 256 : 128;  // keys per online-softmax step of the kernel
    const int cap = decode_auto_splits(Nk);
    int best = cap;
    long long best_cost = LLONG_MAX;
    for (int sp = 1; sp <= cap; ++sp) {
        const long long chunk = (Nk + sp - 1) / sp;
        const long long waves = (bh * sp + resident - 1) / resident;
        const long long cost = waves * ((chunk + piece - 1) / piece * piece + 128);
        if (cost < best_cost) {
            best_cost = cost;
            best = sp;
        }
    }
    *splits = best;
    return FA_OK;
}

// Paged decode, automatic splits.  The lengths live on the device, so the host
// plans for the longest possible sequence (max_pages * page).  The tensor-core
// kernel is persistent: items = B * Hkv * (head groups) * splits are dealt to
// the SMs round-robin.  Its cost model is waves * (1/splits + 0.02): a split
// is a share of the sequence plus a fixed per-item overhead.  It picks the
// best of 1..16 splits with at least 128 keys each.  The general kernel uses
// the contiguous decode's rule.
int paged_auto_splits(int B, int Hq, int Hkv, int max_len, int num_sms, bool mma) {
    if (!mma) return decode_auto_splits(max_len);
    const int g = Hq / Hkv;
    const int nh = g <= 4 ? 4 : (g <= 8 ? 8 : 16);
    const long long base = (long long)B * Hkv * ((g + nh - 1) / nh);
    int best = 1;
    double best_cost = 1e30;
    for (int sp = 1; sp <= 16 && (sp == 1 || (long long)sp * 128 <= max_len); ++sp) {
        const long long waves = (base * sp + num_sms - 1) / num_sms;
        const double cost = (double)waves * (1.0 / sp + 0.02);
        if (cost < best_cost - 1e-12) {
            best_cost = cost;
            best = sp;
        }
    }
    return best;
}

size_t decode_ws_bytes(int B, int H, int d, int splits) {
    const size_t parts = (size_t)B * H * splits;
    return parts * d * 4 + ((parts * 4 + 255) & ~(size_t)255);
}

// Watchdog self-test: one thread waits on an mbarrier that nothing ever
// arrives on.  The bounded wait gives up after `timeout_ns`, records
// FA_ERR_TIMEOUT at kSiteProbe in the error word and the kernel returns.
__global__ void selftest_wait_kernel(DevError* err, uint64_t timeout_ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x != 0) return;
    abort_flag = 0;
    const uint32_t b = smem_u32(&bar);
    mbar_init(b, 1);
    fence_mbar_init();
    const WaitCtl ctl{err, timeout_ns, &abort_flag};
    mbar_wait(b, 0, ctl, kSiteProbe);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_version(void) { return 100; }

uint64_t fa_set_wait_timeout_ns(uint64_t ns) {
    if (ns < 1000000ull) ns = 1000000ull;
    return g_timeout_ns.exchange(ns);
}

const char* fa_status_string(int st) {
    switch (st) {
        case FA_OK: return "ok";
        case FA_ERR_INVALID_ARG: return "invalid argument";
        case FA_ERR_UNSUPPORTED: return "unsupported shape (d must be 64 or 128)";
        case FA_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
        case FA_ERR_WORKSPACE: return "workspace missing or too small";
        case FA_ERR_CUDA: return "CUDA call failed";
        case FA_ERR_TIMEOUT: return "device-side wait timed out";
        default: return "unknown status";
    }
}

}  // extern "C"

namespace {
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq, int Nk,
             int d, float scale, int causal, int window, const int* lens_q, const int* lens_k, void* stream) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
    int st = check_shape(B, H, Nq, Nk, d);
    if (st != FA_OK) return st;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FA_ERR_ALIGNMENT;
    if ((lens_q && !aligned4(lens_q)) || (lens_k && !aligned4(lens_k))) return FA_ERR_ALIGNMENT;
    FwdLaunch a;
    st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    const int BH = B * H;
    if (make_map(&a.map_q, q, BH, Nq, d) || make_map(&a.map_k, k, BH, Nk, d) ||
        make_map(&a.map_v, v, BH, Nk, d))
        return FA_ERR_CUDA;
    a.o = o;
    a.lse = lse;
    a.B = B;
    a.H = H;
    a.Nq = Nq;
    a.Nk = Nk;
    a.d = d;
    a.scale = scale;
    a.causal = causal;
    a.window = window;
    a.lens_q = lens_q;
    a.lens_k = lens_k;
    a.timeout_ns = g_timeout_ns.load();
    return launch_fwd(a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
}  // namespace

extern "C" {

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
           int Nk, int d, float scale, int causal, void* stream) {
    return fwd_impl(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, 0, nullptr, nullptr, stream);
}

int fa_work_schedule(int n_items, int chunk_items, int grid, int per_chunk, int* owner) {
    if (n_items < 0 || chunk_items < 1 || grid < 1 || (n_items > 0 && !owner)) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < n_items; ++i) owner[i] = -1;
    for (int c = 0; c < grid; ++c) {
        ItemSeq q;
        for (int w = next_chunked_item(q, n_items, chunk_items, grid, c, per_chunk != 0); w < n_items;
             w = next_chunked_item(q, n_items, chunk_items, grid, c, per_chunk != 0)) {
            if (w < 0 || owner[w] != -1) return FA_ERR_INVALID_ARG;
            owner[w] = c;
        }
    }
    return FA_OK;
}

int fa_fwd_tile_rows(int B, int H, int Nq, int Nk, int d, int causal) {
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    int st = check_shape(B, H, Nq, Nk, d);
    if (st != FA_OK) return st;
    FwdLaunch a;
    st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    a.B = B;
    a.H = H;
    a.Nq = Nq;
    a.Nk = Nk;
    a.d = d;
    a.causal = causal;
    return fwd_use_split(a) ? 128 : kFwdRowsPerCta;
}

int fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, const int* seqlens_q,
                  const int* seqlens_k, int B, int H, int Nq, int Nk, int d, float scale, int causal, void* stream) {
    if (!seqlens_q || !seqlens_k) return FA_ERR_INVALID_ARG;
    return fwd_impl(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, 0, seqlens_q, seqlens_k, stream);
}

int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
                  int Nk, int d, float scale, int window, void* stream) {
    if (window < 1) return FA_ERR_INVALID_ARG;
    return fwd_impl(q, k, v, o, lse, B, H, Nq, Nk, d, scale, 1, window, nullptr, nullptr, stream);
}

size_t fa_bwd_workspace_bytes(int B, int H, int Nq, int Nk, int d) {
    if (check_shape(B, H, Nq, Nk, d) != FA_OK) return 0;
    return bwd_ws_bytes(B, H, Nq, d);
}

size_t fa_bwd_fused_workspace_bytes(int B, int H, int Nq, int Nk, int d) {
    if (check_shape(B, H, Nq, Nk, d) != FA_OK || d != 128) return 0;
    return bwd_ws_bytes(B, H, Nq, d) + (((size_t)B * H * Nq * d * 4 + 255) & ~(size_t)255);
}

}  // extern "C"

namespace {

// Shared checks of the backward steps.  Pointers that a step does not use are
// passed as `used = false` and not checked.
int bwd_prepare(BwdLaunch* a, const void* q, const void* k, const void* v, const void* o, const float* lse,
                const float* delta, const void* dO, void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk,
                int d, float scale, int causal, bool need_maps) {
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
    int st = check_shape(B, H, Nq, Nk, d);
    if (st != FA_OK) return st;
    const void* ptrs[] = {q, k, v, o, lse, delta, dO, dq, dk, dv};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return FA_ERR_ALIGNMENT;
    st = device_state(&a->err, &a->num_sms);
    if (st != FA_OK) return st;
    const int BH = B * H;
    if (need_maps && (make_map(&a->map_q, q, BH, Nq, d) || make_map(&a->map_k, k, BH, Nk, d) ||
                      make_map(&a->map_v, v, BH, Nk, d) || make_map(&a->map_do, dO, BH, Nq, d)))
        return FA_ERR_CUDA;
    if (need_maps && d == 128 && (make_map(&a->map_q2, q, BH, Nq, d, 64) || make_map(&a->map_do2, dO, BH, Nq, d, 64)))
        return FA_ERR_CUDA;
    a->q = q;
    a->k = k;
    a->o = o;
    a->dO = dO;
    a->lse = lse;
    a->dq = dq;
    a->dk = dk;
    a->dv = dv;
    a->delta = const_cast<float*>(delta);
    a->dqacc = nullptr;
    a->B = B;
    a->H = H;
    a->Nq = Nq;
    a->Nk = Nk;
    a->d = d;
    a->scale = scale;
    a->causal = causal;
    a->window = 0;
    a->lens_q = nullptr;
    a->lens_k = nullptr;
    a->timeout_ns = g_timeout_ns.load();
    return FA_OK;
}

int launched(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

int bwd_impl(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
             void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale, int causal,
             int window, const int* lens_q, const int* lens_k, void* workspace, size_t workspace_bytes,
             void* stream, bool fused = false) {
    if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
    if ((lens_q && !aligned4(lens_q)) || (lens_k && !aligned4(lens_k))) return FA_ERR_ALIGNMENT;
    int st = check_shape(B, H, Nq, Nk, d);
    if (st != FA_OK) return st;
    if (fused && d != 128) return FA_ERR_UNSUPPORTED;
    const size_t ws_need = fused ? fa_bwd_fused_workspace_bytes(B, H, Nq, Nk, d) : bwd_ws_bytes(B, H, Nq, d);
    if (!workspace || workspace_bytes < ws_need) return FA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    BwdLaunch a;
    st = bwd_prepare(&a, q, k, v, o, lse, static_cast<float*>(workspace), dO, dq, dk, dv, B, H, Nq, Nk, d,
                     scale, causal, true);
    if (st != FA_OK) return st;
    a.window = window;
    a.lens_q = lens_q;
    a.lens_k = lens_k;
    cudaStream_t s = (cudaStream_t)stream;
    if (fused) {  // the fp32 dQ accumulator follows D in the workspace
        a.dqacc = reinterpret_cast<float*>(static_cast<char*>(workspace) + bwd_ws_bytes(B, H, Nq, d));
        if ((st = launched(launch_bwd_pre(a, s))) != FA_OK) return st;
        return launched(launch_bwd_fused(a, s));
    }
    if ((st = launched(launch_bwd_pre(a, s))) != FA_OK) return st;
    if ((st = launched(launch_bwd_dkdv(a, s, true))) != FA_OK) return st;
    return launched(launch_bwd_dq(a, s, true));
}

}  // namespace

extern "C" {

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
           void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale, int causal,
           void* workspace, size_t workspace_bytes, void* stream) {
    return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, causal, 0, nullptr, nullptr,
                    workspace, workspace_bytes, stream);
}

int fa_bwd_fused(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                 void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                 void* workspace, size_t workspace_bytes, void* stream) {
    return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, causal, 0, nullptr, nullptr,
                    workspace, workspace_bytes, stream, true);
}

int fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                  void* dq, void* dk, void* dv, const int* seqlens_q, const int* seqlens_k, int B, int H, int Nq,
                  int Nk, int d, float scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
    if (!seqlens_q || !seqlens_k) return FA_ERR_INVALID_ARG;
    return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, causal, 0, seqlens_q, seqlens_k,
                    workspace, workspace_bytes, stream);
}

int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                  void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale, int window,
                  void* workspace, size_t workspace_bytes, void* stream) {
    if (window < 1) return FA_ERR_INVALID_ARG;
    return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, 1, window, nullptr, nullptr,
                    workspace, workspace_bytes, stream);
}

int fa_bwd_preprocess(const void* o, const void* dO, float* delta, int B, int H, int Nq, int d, void* stream) {
    if (!o || !dO || !delta) return FA_ERR_INVALID_ARG;
    BwdLaunch a;
    int st = bwd_prepare(&a, nullptr, nullptr, nullptr, o, nullptr, delta, dO, nullptr, nullptr, nullptr, B, H,
                         Nq, 1, d, 1.f, 0, false);
    if (st != FA_OK) return st;
    return launched(launch_bwd_pre(a, (cudaStream_t)stream));
}

int fa_bwd_dkdv(const void* q, const void* k, const void* v, const float* lse, const float* delta,
                const void* dO, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale, int causal,
                void* stream) {
    if (!q || !k || !v || !lse || !delta || !dO || !dk || !dv) return FA_ERR_INVALID_ARG;
    BwdLaunch a;
    int st = bwd_prepare(&a, q, k, v, nullptr, lse, delta, dO, nullptr, dk, dv, B, H, Nq, Nk, d, scale, causal,
                         true);
    if (st != FA_OK) return st;
    return launched(launch_bwd_dkdv(a, (cudaStream_t)stream));
}

int fa_bwd_dkdv_pair(const void* q, const void* k, const void* v, const float* lse, const float* delta,
                     const void* dO, void* dk, void* dv, int B, int H, int Nq, int Nk, int d, float scale,
                     int causal, void* stream) {
    if (!q || !k || !v || !lse || !delta || !dO || !dk || !dv) return FA_ERR_INVALID_ARG;
    if (d == 64) return FA_ERR_UNSUPPORTED;  // other d: the shape check below
    BwdLaunch a;
    int st = bwd_prepare(&a, q, k, v, nullptr, lse, delta, dO, nullptr, dk, dv, B, H, Nq, Nk, d, scale, causal,
                         true);
    if (st != FA_OK) return st;
    return launched(launch_bwd_dkdv_pair(a, (cudaStream_t)stream));
}

int fa_bwd_dq(const void* q, const void* k, const void* v, const float* lse, const float* delta, const void* dO,
              void* dq, int B, int H, int Nq, int Nk, int d, float scale, int causal, void* stream) {
    if (!q || !k || !v || !lse || !delta || !dO || !dq) return FA_ERR_INVALID_ARG;
    BwdLaunch a;
    int st = bwd_prepare(&a, q, k, v, nullptr, lse, delta, dO, dq, nullptr, nullptr, B, H, Nq, Nk, d, scale,
                         causal, true);
    if (st != FA_OK) return st;
    return launched(launch_bwd_dq(a, (cudaStream_t)stream));
}

size_t fa_decode_workspace_bytes(int B, int H, int Nk, int d, int num_splits) {
    if (check_shape(B, H, 1, Nk, d) != FA_OK || num_splits > 256) return 0;
    const int s = num_splits <= 0 ? decode_auto_splits(Nk) : num_splits;
    return decode_ws_bytes(B, H, d, s);
}

}  // extern "C"

namespace {

// Tensor maps of the tensor-core paged decode (d = 128): q, and K/V as pages.
int paged_mma_maps(PagedDecodeLaunch& a) {
    const int d = a.d, page_size = a.page;
    const cuuint64_t qd[3] = {(cuuint64_t)d, (cuuint64_t)a.B * a.Hq, 1};
    const cuuint64_t qs[2] = {(cuuint64_t)d * 2, (cuuint64_t)a.B * a.Hq * d * 2};
    const cuuint32_t qb[3] = {64, 16, 1};
    const cuuint64_t kd[4] = {(cuuint64_t)d, (cuuint64_t)page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
    const cuuint64_t ks[3] = {(cuuint64_t)d * 2, (cuuint64_t)page_size * d * 2,
                              (cuuint64_t)a.Hkv * page_size * d * 2};
    const cuuint32_t kb[4] = {64, (cuuint32_t)page_box_rows(page_size), 1, 1};
    // V: the feature dimension as (64, half) so one box holds a page's rows of both halves
    const cuuint64_t vd[5] = {64, (cuuint64_t)page_size, 2, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
    const cuuint64_t vs[4] = {(cuuint64_t)d * 2, 128, (cuuint64_t)page_size * d * 2,
                              (cuuint64_t)a.Hkv * page_size * d * 2};
    const cuuint32_t vb[5] = {64, (cuuint32_t)page_box_rows(page_size), 2, 1, 1};
    // d = 64: a row is one 128-byte swizzle row, so V takes the same 4-D form as K.  d = 128 with
    // 8-row boxes: K takes V's 5-D form too (one copy per box for both feature halves; the kernel
    // addresses the halves 1 KB apart and the 8-row groups 2 KB apart)
    const bool k5 = d == 128 && page_box_rows(page_size) == 8;
    if (make_map_nd(&a.map_q, a.q, 3, qd, qs, qb) ||
        (k5 ? make_map_nd(&a.map_k, a.kp, 5, vd, vs, vb) : make_map_nd(&a.map_k, a.kp, 4, kd, ks, kb)) ||
        (d == 128 ? make_map_nd(&a.map_v, a.vp, 5, vd, vs, vb) : make_map_nd(&a.map_v, a.vp, 4, kd, ks, kb)))
        return FA_ERR_CUDA;
    return FA_OK;
}

// Contiguous decode (fa_decode, fa_decode_noalloc) with d = 128 and Nk a multiple of 128 runs on the
// tensor-core paged kernel: the cache [B, H, Nk, d] is the paged layout with one page of Nk tokens per
// sequence (page b of sequence b, implicit in the kernel), one kv head per query head.  Its TMA stages
// read the cache at ~6.8 TB/s against ~6.3 TB/s for the 16-byte-load kernel.  Other shapes are faster
// on the 16-byte-load kernel (measured at B=32, H=32, 16 splits): with one query head per kv head
// every work item is a split of two 128-key stages, and the kernel's fixed cost per item and per
// stage, which d = 128 hides behind 64 KB of cache per stage, shows at d = 64 (4.0 against 5.8 TB/s
// at Nk = 4096) and on a ragged last stage (6.0 against 6.2 TB/s at Nk = 4000).  Returns false when
// the shape takes the 16-byte-load kernel.
bool contiguous_on_mma(int Nk, int d) { return d == 128 && Nk % 128 == 0 && paged_mma_ok(d, Nk); }

int launch_contiguous_on_mma(const void* q, const void* kcache, const void* vcache, void* o, float* lse, int B,
                             int H, int Nk, int d, float scale, int splits, float* part_o, void* stream) {
    PagedDecodeLaunch a;
    int st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    a.mma = true;
    a.q = q;
    a.kp = kcache;
    a.vp = vcache;
    a.table = nullptr;
    a.lens = nullptr;
    a.o = o;
    a.lse = lse;
    a.part_o = part_o;
    a.part_lse = part_o + (size_t)B * H * splits * d;  // the layout of the fa_decode workspace
    a.B = B;
    a.Hq = H;
    a.Hkv = H;
    a.page = Nk;
    a.max_pages = 1;
    a.num_pages = B;
    a.d = d;
    a.splits = splits;
    a.scale = scale;
    a.timeout_ns = g_timeout_ns.load();
    st = paged_mma_maps(a);
    if (st != FA_OK) return st;
    return launch_decode_paged(a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

int fa_decode(const void* q, const void* kcache, const void* vcache, void* o, float* lse, int B, int H,
              int Nk, int d, float scale, int num_splits, void* workspace, size_t workspace_bytes,
              void* stream) {
    if (!q || !kcache || !vcache || !o) return FA_ERR_INVALID_ARG;
    if (!scale_ok(scale) || num_splits > 256) return FA_ERR_INVALID_ARG;
    int st = check_shape(B, H, 1, Nk, d);
    if (st != FA_OK) return st;
    if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(o) ||
        (lse && !aligned16(lse)))
        return FA_ERR_ALIGNMENT;
    // automatic: the tensor-core path reads best with the most splits its length allows; the
    // CUDA-core kernel takes the wave rule above.  Both stay within decode_auto_splits(Nk), the
    // count fa_decode_workspace_bytes sizes for.
    int splits = num_splits <= 0 ? decode_auto_splits(Nk) : num_splits;
    if (num_splits <= 0 && !contiguous_on_mma(Nk, d)) {
        st = decode_wave_splits(B, H, Nk, d, &splits);
        if (st != FA_OK) return st;
    }
    if (!workspace || workspace_bytes < decode_ws_bytes(B, H, d, splits)) return FA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    if (contiguous_on_mma(Nk, d))
        return launch_contiguous_on_mma(q, kcache, vcache, o, lse, B, H, Nk, d, scale, splits,
                                        static_cast<float*>(workspace), stream);
    st = device_state(nullptr, nullptr);
    if (st != FA_OK) return st;
    DecodeLaunch a;
    a.q = q;
    a.kc = kcache;
    a.vc = vcache;
    a.o = o;
    a.lse = lse;
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = a.part_o + (size_t)B * H * splits * d;
    a.B = B;
    a.H = H;
    a.Nk = Nk;
    a.d = d;
    a.splits = splits;
    a.chunk = (Nk + splits - 1) / splits;
    a.scale = scale;
    return launch_decode(a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_decode_paged_workspace_bytes(int B, int Hq, int d, int num_splits) {
    if (B < 1 || Hq < 1 || (d != 64 && d != 128) || num_splits > 256) return 0;
    return decode_ws_bytes(B, Hq, d, num_splits <= 0 ? 16 : num_splits);  // automatic: at most 16
}

int fa_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                    const int* seq_lens, void* o, float* lse, int B, int Hq, int Hkv, int page_size,
                    int max_pages, int num_pages, int d, float scale, int num_splits, void* workspace,
                    size_t workspace_bytes, void* stream) {
    if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !o) return FA_ERR_INVALID_ARG;
    if (!scale_ok(scale) || num_splits > 256) return FA_ERR_INVALID_ARG;
    if (B < 1 || Hq < 1 || Hkv < 1 || page_size < 1 || max_pages < 1 || num_pages < 1) return FA_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size > 0x7FFFFFFFll || (long long)B * Hq > (1ll << 24)) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) || (lse && !aligned16(lse)) ||
        (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
        return FA_ERR_ALIGNMENT;
    PagedDecodeLaunch a;
    int st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    a.mma = paged_mma_ok(d, page_size);
    if (num_splits <= 0)
        num_splits = paged_auto_splits(B, Hq, Hkv, max_pages * page_size, a.num_sms, a.mma);
    if (!workspace || workspace_bytes < decode_ws_bytes(B, Hq, d, num_splits)) return FA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    a.q = q;
    a.kp = k_pages;
    a.vp = v_pages;
    a.table = block_table;
    a.lens = seq_lens;
    a.o = o;
    a.lse = lse;
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = a.part_o + (size_t)B * Hq * num_splits * d;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.page = page_size;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.d = d;
    a.splits = num_splits;
    a.scale = scale;
    if (a.mma) {
        a.timeout_ns = g_timeout_ns.load();
        st = paged_mma_maps(a);
        if (st != FA_OK) return st;
    }
    return launch_decode_paged(a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_fwd_fp8_workspace_bytes(int B, int H, int Nk, int d) {
    if (B < 1 || H < 1 || Nk < 1 || d != 128 || (long long)B * H > (1ll << 24)) return 0;
    const size_t nk_pad = ((size_t)Nk + 15) & ~(size_t)15;
    return (((size_t)B * H * 128 * nk_pad) + 255) & ~(size_t)255;
}

int fa_fwd_fp8(const void* q, const void* k, const void* v, const float* q_scale, const float* k_scale,
               const float* v_scale, void* o, float* lse, int B, int H, int Nq, int Nk, int d, float scale,
               int causal, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !k || !v || !q_scale || !k_scale || !v_scale || !o || !lse) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
    int st = check_shape(B, H, Nq, Nk, d);
    if (st != FA_OK) return st;
    if (d != 128) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
        !aligned4(q_scale) || !aligned4(k_scale) || !aligned4(v_scale))
        return FA_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < fa_fwd_fp8_workspace_bytes(B, H, Nk, d)) return FA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    Fp8FwdLaunch a;
    st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    const cuuint64_t BH = (cuuint64_t)B * H;
    const int nk_pad = (Nk + 15) & ~15;
    const cuuint32_t box[3] = {128, 128, 1};
    const cuuint64_t qd[3] = {128, (cuuint64_t)Nq, BH}, qs[2] = {128, (cuuint64_t)Nq * 128};
    const cuuint64_t kd[3] = {128, (cuuint64_t)Nk, BH}, ks[2] = {128, (cuuint64_t)Nk * 128};
    const cuuint64_t vd[3] = {(cuuint64_t)nk_pad, 128, BH}, vs[2] = {(cuuint64_t)nk_pad, (cuuint64_t)nk_pad * 128};
    if (make_map_nd(&a.map_q, q, 3, qd, qs, box, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
        make_map_nd(&a.map_k, k, 3, kd, ks, box, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
        make_map_nd(&a.map_vt, workspace, 3, vd, vs, box, CU_TENSOR_MAP_DATA_TYPE_UINT8))
        return FA_ERR_CUDA;
    a.v = v;
    a.vt = workspace;
    a.o = o;
    a.lse = lse;
    a.q_scale = q_scale;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.B = B;
    a.H = H;
    a.Nq = Nq;
    a.Nk = Nk;
    a.Nk_pad = nk_pad;
    a.scale = scale;
    a.causal = causal;
    a.timeout_ns = g_timeout_ns.load();
    return launch_fwd_fp8(a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"

// ---------------------------------------------------------------- rotary positions and the 8-bit cache
namespace {

// Strides of a [B, H, N, d] tensor: d innermost, the others multiples of 8 elements (16 bytes); that of a
// dimension of size 1 is not used (set to 0).
int check_strides(long long* sb, long long* sh, long long* sn, int B, int H, int N) {
    if (B == 1) *sb = 0;
    if (H == 1) *sh = 0;
    if (N == 1) *sn = 0;
    if (*sb < 0 || *sh < 0 || *sn < 0) return FA_ERR_INVALID_ARG;
    if ((*sb | *sh | *sn) & 7) return FA_ERR_ALIGNMENT;
    return FA_OK;
}

// Whether no two elements of such a tensor share an address.
bool strides_distinct(long long sb, long long sh, long long sn, int B, int H, int N, int d) {
    std::pair<long long, int> s[3] = {{sb, B}, {sh, H}, {sn, N}};
    std::sort(s, s + 3);
    long long extent = d;
    for (const auto& x : s) {
        if (x.second == 1) continue;
        if (x.first < extent) return false;
        extent += x.first * (x.second - 1);
    }
    return true;
}

int check_rotation(int d, int rot, int interleaved, float magnitude) {
    if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(magnitude) || rot < 1 || rot > d) return FA_ERR_INVALID_ARG;
    return rot % 16 ? FA_ERR_UNSUPPORTED : FA_OK;
}

constexpr long long kMaxCacheTokens = 1ll << 30;  // of one sequence: token arithmetic stays in int

// Sizes of the paged 8-bit cache that its three entry points share.
int check_cache(int B, int Hkv, int page, int sb, int max_pages, int num_pages, int d) {
    if (B < 1 || Hkv < 1 || page < 1 || sb < 1 || max_pages < 1 || num_pages < 1) return FA_ERR_INVALID_ARG;
    if (page % sb) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (sb > 128) return FA_ERR_UNSUPPORTED;
    if ((long long)max_pages * page > kMaxCacheTokens || (long long)B * Hkv > (1ll << 24)) return FA_ERR_UNSUPPORTED;
    // cache rows (num_pages * Hkv * page) are counted in 32 bits
    if ((long long)num_pages * Hkv > 0xFFFFFFFEll / page) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

int g_fp8_blocks[kMaxDevices][2][3] = {};  // resident CTAs per SM of the 8-bit decode, by device, d and tile rows

constexpr int kFp8MostWorkers = 1024;  // bounds the workspace; four CTAs (d = 64) on each of 152 SMs are 608

// CTAs that the 8-bit decode shares its steps among: as many as run at once.
int fp8_workers(int d, int tile, int num_sms, int* workers) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    int& c = g_fp8_blocks[dev][d == 128 ? 1 : 0][tile == 8 ? 0 : tile == 16 ? 1 : 2];
    if (!c) {
        int b = 0;
        if (decode_fp8_blocks_per_sm(d, tile, &b) != cudaSuccess || b < 1) return FA_ERR_CUDA;
        c = b;
    }
    *workers = std::min(kFp8MostWorkers, num_sms * c);
    return FA_OK;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace of the 8-bit decode: partial outputs and LSEs of every segment (at most one more per worker than there are
// items), the sequences' first steps, and with weights the scores of every row and token.
struct Fp8Workspace {
    size_t part_lse, prefix, lse2, scores, bytes;
};
Fp8Workspace fp8_workspace(int B, int Hq, int Hkv, int Nq, int d, long long max_tokens, bool weights) {
    const int rows = Hq / Hkv * Nq, tile = fp8_tile_rows(rows);
    const size_t slots = (size_t)kFp8MostWorkers + (size_t)B * Hkv * ((rows + tile - 1) / tile);
    Fp8Workspace w;
    w.part_lse = align256(slots * tile * d * 4);
    w.prefix = w.part_lse + align256(slots * tile * 4);
    w.lse2 = w.prefix + align256(((size_t)B + 1) * 8);
    w.scores = w.lse2 + (weights ? align256((size_t)B * Hq * Nq * 4) : 0);
    w.bytes = w.scores + (weights ? align256((size_t)B * Hkv * ((rows + 3) & ~3) * (size_t)max_tokens * 4) : 0);
    return w;
}

// Workspace of the block selection: exact keys and scores of every block of the table.
struct SelectWorkspace {
    size_t scores, bytes;
};
SelectWorkspace select_workspace(int B, int Hkv, long long max_blocks) {
    const size_t bh = (size_t)B * Hkv;
    SelectWorkspace w;
    w.scores = align256(bh * (size_t)max_blocks * 8);
    w.bytes = w.scores + align256(bh * (size_t)max_blocks * 4);
    return w;
}

// Workspace of the bf16 row decode: partial outputs and LSEs of every segment (at most one more per CTA than there are
// items), and the first and last CTA of every item.
struct RowsWorkspace {
    size_t part_lse, ends, bytes;
};
RowsWorkspace rows_workspace(int B, int Hq, int Hkv, int Nq, int d, int joint = 0, bool by_prefix = false) {
    const int rows = Hq / Hkv * Nq, tile = by_prefix ? 8 : rows_tile(joint ? joint : rows);
    const size_t items = ((size_t)B + (joint + tile - 1) / tile) * Hkv * ((rows + tile - 1) / tile), slots = (size_t)kRowsMostWorkers + items;
    RowsWorkspace w;
    w.part_lse = align256(slots * tile * d * 4);
    w.ends = w.part_lse + align256(slots * tile * 4);
    w.bytes = w.ends + align256(items * 8);
    return w;
}

// Workspace of the shared prefix: the same of (kv head, tile of the batch's query rows) items.  Its parts are stored 32 bytes
// at a time; a caller's workspace has 16-byte alignment, so the call may skip kPrefixSkip bytes at its start.
constexpr size_t kPrefixSkip = 16;
struct PrefixWorkspace {
    int tiles, tile_rows;
    size_t part_lse, ends, bytes;
};
PrefixWorkspace prefix_workspace(int B, int Hq, int Hkv, int Nq, int d) {
    const long long rows = (long long)B * (Hq / Hkv) * Nq;
    PrefixWorkspace w;
    w.tile_rows = rows <= 128 ? 128 : 256;
    w.tiles = (int)((rows + w.tile_rows - 1) / w.tile_rows);
    const size_t items = (size_t)Hkv * w.tiles, slots = (size_t)kPrefixMostWorkers + items;
    w.part_lse = align256(slots * w.tile_rows * d * 4);
    w.ends = w.part_lse + align256(slots * w.tile_rows * 4);
    w.bytes = w.ends + align256(items * 8);
    return w;
}

// Where the prefix's kernel takes the own tokens too, 8 query rows of a sequence and kv head at a time: up to 16 rows (64
// sequences, 8 kv heads, d = 128, 1000 shared tokens and up to 20 own ones: 36.3 us apart, 31.5 together; 16 sequences 25.8 and
// 19.2), and up to 32 where there are few (sequence, kv head) pairs to read four times (128 pairs of 24 rows 26.2 and 19.5; 512
// pairs of 32 rows 41.2 and 53.5).
bool prefix_takes_own(int B, int Hq, int Hkv, int Nq) {
    const int rows = Hq / Hkv * Nq;
    return rows <= 16 || (rows <= 32 && (long long)B * Hkv <= 128);
}

// Query rows of all sequences where decode_rows takes the prefix too, 0 where it does not: it reads the prefix once for each
// 32 of them, which saves the other kernel's start and end where that is little work.  Measured with 8 kv heads, d = 128, up to 100
// own tokens, against the prefix's kernel with the own tokens in it (calls back to back on 24 sets of inputs): 4 rows of a sequence, 32
// rows in all, 1000 shared tokens 11.7 and 13.6 us, 2000 15.0 and 15.5, 4000 16.4 and 16.9; 64 rows 13.4 and 14.2, 2000 16.3 and
// 16.0; 128 rows, 250 tokens 14.4 and 14.6, 500 15.3 and 15.5; 16 rows of a sequence, 128 in all, 500 tokens 13.2 and 14.2, 1000 15.6
// and 14.8.  Far beyond the limits the prefix's kernel gains (32 rows, 8000 tokens 20.2 and 17.2; 64 rows 25.5 and 18.2).  With fewer
// heads or d = 64 they meet where tokens x heads x d does.  tokens: of the table, since the host does not know how many are shared,
// so that a batch in a wide table has the prefix's kernel whatever it shares; 0: where any table of such a batch would do.
int joint_rows(int B, int Hq, int Hkv, int Nq, int d, long long tokens) {
    const long long rows = (long long)B * (Hq / Hkv) * Nq, tiles = (rows + 31) / 32;
    if (rows > 128 || Hq / Hkv * Nq > 32) return 0;
    const long long most = (tiles <= 2 || Hq / Hkv * Nq > 8 ? 4096ll : 2048ll) * 8 * 128;  // elements of keys
    return tokens <= most / (tiles * Hkv * d) ? (int)rows : 0;
}

bool rows_sizes_ok(int B, int Hq, int Hkv, int Nq, int d) {
    return B >= 1 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && Nq >= 1 && Nq <= 16 && (d == 64 || d == 128) &&
           (long long)B * Hq <= (1ll << 24);
}

// Checks and fields that the attention over blocks and the one with a shared prefix have in common.
int rows_prepare(DecodeRowsLaunch& a, const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                 const int* seq_lens, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int page_size, int block,
                 int max_pages, int num_pages, int d, float scale, bool by_prefix = false) {
    if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !o) return FA_ERR_INVALID_ARG;
    if (!scale_ok(scale) || Hq < 1 || Nq < 1) return FA_ERR_INVALID_ARG;
    int st = check_cache(B, Hkv, page_size, block, max_pages, num_pages, d);
    if (st != FA_OK) return st;
    if (Hq % Hkv) return FA_ERR_INVALID_ARG;
    if (!rows_sizes_ok(B, Hq, Hkv, Nq, d)) return FA_ERR_UNSUPPORTED;
    // steps of 64 keys over all sequences, kv heads and row tiles, and two more for each of these, are counted in 31 bits
    const int rows = Hq / Hkv * Nq, tile = by_prefix ? 8 : rows_tile(rows);
    if (((long long)B + 4) * Hkv * ((rows + tile - 1) / tile) > 0x7FFFFFFFll / (((long long)max_pages * page_size + block + 63) / 64 + 2))
        return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) || !aligned4(block_table) ||
        !aligned4(seq_lens) || !aligned4(lse))
        return FA_ERR_ALIGNMENT;
    if (o == q) return FA_ERR_INVALID_ARG;  // other CTAs may still read the row that one writes
    a.q = q;
    a.kp = k_pages;
    a.vp = v_pages;
    a.table = block_table;
    a.lens = seq_lens;
    a.list = nullptr;
    a.shared = nullptr;
    a.o = o;
    a.lse = lse;
    a.pre_o = a.pre_lse = nullptr;
    a.pre_ends = nullptr;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Nq = Nq;
    a.page = page_size;
    a.block = block;
    a.keep = 0;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.d = d;
    a.pre_workers = a.pre_tiles = a.pre_rows = a.joint = 0;
    a.merge_only = false;
    a.scale = scale;
    return FA_OK;
}

void rows_place(DecodeRowsLaunch& a, char* base) {
    const RowsWorkspace w = rows_workspace(a.B, a.Hq, a.Hkv, a.Nq, a.d, a.joint, a.merge_only);
    a.part_o = reinterpret_cast<float*>(base);
    a.part_lse = reinterpret_cast<float*>(base + w.part_lse);
    a.ends = reinterpret_cast<int*>(base + w.ends);
}

}  // namespace

extern "C" {

int fa_rope_table(const double* inv_freq, int n, uint64_t* turns) {
    if (!inv_freq || !turns || n < 1) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(inv_freq[i])) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        const double t = std::fabs(inv_freq[i]) / 6.283185307179586;  // turns per position; whole turns drop out
        const double f = t - std::floor(t);                           // [0, 1), exact
        // 2^64 f in two 32-bit steps, each exact in a double
        const double hi = std::floor(f * 4294967296.0), lo = std::nearbyint((f * 4294967296.0 - hi) * 4294967296.0);
        const uint64_t u = ((uint64_t)hi << 32) + (uint64_t)lo;
        turns[i] = inv_freq[i] < 0 ? 0 - u : u;  // modulo a turn; 1 - f would lose the low bits of a small f
    }
    return FA_OK;
}

int fa_rope(const void* x, void* y, long long x_sb, long long x_sh, long long x_sn, long long y_sb, long long y_sh,
            long long y_sn, const int* positions, const uint64_t* turns, int B, int H, int N, int d, int rot,
            int interleaved, float magnitude, int inverse, void* stream) {
    if (!x || !y || !turns || B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
    if (inverse != 0 && inverse != 1) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    int st = check_rotation(d, rot, interleaved, magnitude);
    if (st != FA_OK) return st;
    if ((long long)B * N > 0x7FFFFFFFll || (long long)B * H > (1ll << 24)) return FA_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(y) || !aligned16(turns) || (positions && !aligned4(positions)))
        return FA_ERR_ALIGNMENT;
    if ((st = check_strides(&x_sb, &x_sh, &x_sn, B, H, N)) != FA_OK) return st;
    if ((st = check_strides(&y_sb, &y_sh, &y_sn, B, H, N)) != FA_OK) return st;
    if (!strides_distinct(y_sb, y_sh, y_sn, B, H, N, d)) return FA_ERR_INVALID_ARG;
    if (x == y && (x_sb != y_sb || x_sh != y_sh || x_sn != y_sn)) return FA_ERR_INVALID_ARG;
    RopeLaunch a;
    st = device_state(nullptr, &a.num_sms);
    if (st != FA_OK) return st;
    a.x = x;
    a.y = y;
    a.xb = x_sb;
    a.xh = x_sh;
    a.xn = x_sn;
    a.yb = y_sb;
    a.yh = y_sh;
    a.yn = y_sn;
    a.positions = positions;
    a.turns = turns;
    a.tokens = (long long)B * N;
    a.H = H;
    a.N = N;
    a.d = d;
    a.rot = rot;
    a.interleaved = interleaved;
    a.inverse = inverse;
    a.magnitude = magnitude;
    return launched(launch_rope(a, (cudaStream_t)stream));
}

int fa_cache_append_fp8(const void* k, const void* v, long long k_sb, long long k_sh, long long k_sn, long long v_sb,
                        long long v_sh, long long v_sn, void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                        const int* block_table, const int* seq_lens, const int* new_lens, const int* positions,
                        const uint64_t* turns, int B, int Hkv, int N, int d, int rot, int interleaved, float magnitude,
                        int page_size, int scale_block, int max_pages, int num_pages, void* stream) {
    if (!k || !v || !k_pages || !v_pages || !k_scale || !v_scale || !block_table || !seq_lens || N < 1)
        return FA_ERR_INVALID_ARG;
    int st = check_cache(B, Hkv, page_size, scale_block, max_pages, num_pages, d);
    if (st != FA_OK) return st;
    if (turns && (st = check_rotation(d, rot, interleaved, magnitude)) != FA_OK) return st;
    if (N > kMaxCacheTokens / 2 || (long long)B * Hkv * N > 0x7FFFFFFFll) return FA_ERR_UNSUPPORTED;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(turns) ||
        !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(block_table) || !aligned4(seq_lens) ||
        !aligned4(new_lens) || !aligned4(positions))
        return FA_ERR_ALIGNMENT;
    if ((st = check_strides(&k_sb, &k_sh, &k_sn, B, Hkv, N)) != FA_OK) return st;
    if ((st = check_strides(&v_sb, &v_sh, &v_sn, B, Hkv, N)) != FA_OK) return st;
    CacheAppendLaunch a;
    st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    a.k = k;
    a.v = v;
    a.kb = k_sb;
    a.kh = k_sh;
    a.kn = k_sn;
    a.vb = v_sb;
    a.vh = v_sh;
    a.vn = v_sn;
    a.kp = static_cast<uint8_t*>(k_pages);
    a.vp = static_cast<uint8_t*>(v_pages);
    a.ks = k_scale;
    a.vs = v_scale;
    a.table = block_table;
    a.lens = seq_lens;
    a.new_lens = new_lens;
    a.positions = positions;
    a.turns = turns;
    a.B = B;
    a.Hkv = Hkv;
    a.N = N;
    a.d = d;
    a.rot = rot;
    a.interleaved = turns ? interleaved : 0;
    a.page = page_size;
    a.sb = scale_block;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.magnitude = magnitude;
    return launched(launch_cache_append(a, (cudaStream_t)stream));
}

size_t fa_decode_paged_fp8_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, int max_tokens, int weights) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Nq < 1 || Nq > 16 || (d != 64 && d != 128) || max_tokens < 1) return 0;
    if (max_tokens > kMaxCacheTokens || (long long)B * Hq > (1ll << 24) || (weights != 0 && weights != 1)) return 0;
    return fp8_workspace(B, Hq, Hkv, Nq, d, max_tokens, weights != 0).bytes;
}

int fa_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                        const float* v_scale, const int* block_table, const int* seq_lens, void* o, float* lse,
                        float* weights, int B, int Hq, int Hkv, int Nq, int page_size, int scale_block, int max_pages,
                        int num_pages, int d, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !block_table || !seq_lens || !o) return FA_ERR_INVALID_ARG;
    if (!scale_ok(scale) || Hq < 1 || Nq < 1) return FA_ERR_INVALID_ARG;
    int st = check_cache(B, Hkv, page_size, scale_block, max_pages, num_pages, d);
    if (st != FA_OK) return st;
    if (Hq % Hkv) return FA_ERR_INVALID_ARG;
    if (Nq > 16 || (long long)B * Hq > (1ll << 24)) return FA_ERR_UNSUPPORTED;
    // steps of 128 tokens over all sequences, kv heads and row tiles are counted in 32 bits per CTA
    const int rows = Hq / Hkv * Nq, tile = fp8_tile_rows(rows);
    if ((long long)B * Hkv * ((rows + tile - 1) / tile) > 0x7FFFFFFFll / (((long long)max_pages * page_size + 127) / 128))
        return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) || !aligned4(k_scale) ||
        !aligned4(v_scale) || !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(lse) || !aligned4(weights))
        return FA_ERR_ALIGNMENT;
    if (o == q) return FA_ERR_INVALID_ARG;  // other CTAs may still read the row that one writes
    PagedDecodeFp8Launch a;
    st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    st = fp8_workers(d, tile, a.num_sms, &a.workers);
    if (st != FA_OK) return st;
    const Fp8Workspace ws = fp8_workspace(B, Hq, Hkv, Nq, d, (long long)max_pages * page_size, weights != nullptr);
    if (!workspace || workspace_bytes < ws.bytes) return FA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    char* base = static_cast<char*>(workspace);
    a.q = q;
    a.kp = static_cast<const uint8_t*>(k_pages);
    a.vp = static_cast<const uint8_t*>(v_pages);
    a.ks = k_scale;
    a.vs = v_scale;
    a.table = block_table;
    a.lens = seq_lens;
    a.o = o;
    a.lse = lse;
    a.weights = weights;
    a.part_o = reinterpret_cast<float*>(base);
    a.part_lse = reinterpret_cast<float*>(base + ws.part_lse);
    a.scores = reinterpret_cast<float*>(base + ws.scores);
    a.prefix = reinterpret_cast<long long*>(base + ws.prefix);
    a.lse2 = reinterpret_cast<float*>(base + ws.lse2);
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Nq = Nq;
    a.page = page_size;
    a.sb = scale_block;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.d = d;
    a.scale = scale;
    return launched(launch_decode_paged_fp8(a, (cudaStream_t)stream));
}

int fa_cache_evict_fp8(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const int* block_table,
                       const int* seq_lens, const float* weights, const int* new_table, int* new_lens,
                       float* new_weights, int* kept, int B, int Hkv, int page_size, int scale_block, int max_pages,
                       int new_max_pages, int num_pages, int d, int keep, int recent, void* stream) {
    if (!k_pages || !v_pages || !k_scale || !v_scale || !block_table || !seq_lens || !weights || !new_table ||
        !new_lens || !new_weights || !kept)
        return FA_ERR_INVALID_ARG;
    int st = check_cache(B, Hkv, page_size, scale_block, max_pages, num_pages, d);
    if (st != FA_OK) return st;
    if (new_max_pages < 1 || keep < 1 || recent < 0 || recent > keep) return FA_ERR_INVALID_ARG;
    if ((long long)new_max_pages * page_size > kMaxCacheTokens) return FA_ERR_UNSUPPORTED;
    if (keep > (long long)new_max_pages * page_size) return FA_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned4(k_scale) || !aligned4(v_scale) ||
        !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(weights) || !aligned4(new_table) ||
        !aligned4(new_lens) || !aligned4(new_weights) || !aligned4(kept))
        return FA_ERR_ALIGNMENT;
    if (new_lens == seq_lens || new_weights == weights) return FA_ERR_INVALID_ARG;  // read while the other is written
    CacheEvictLaunch a;
    st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    a.kp = static_cast<uint8_t*>(k_pages);
    a.vp = static_cast<uint8_t*>(v_pages);
    a.ks = k_scale;
    a.vs = v_scale;
    a.table = block_table;
    a.lens = seq_lens;
    a.weights = weights;
    a.new_table = new_table;
    a.new_lens = new_lens;
    a.new_weights = new_weights;
    a.kept = kept;
    a.B = B;
    a.Hkv = Hkv;
    a.page = page_size;
    a.sb = scale_block;
    a.max_pages = max_pages;
    a.new_max_pages = new_max_pages;
    a.num_pages = num_pages;
    a.d = d;
    a.keep = keep;
    a.recent = recent;
    return launched(launch_cache_evict(a, (cudaStream_t)stream));
}

int fa_cache_append(const void* k, const void* v, long long k_sb, long long k_sh, long long k_sn, long long v_sb,
                    long long v_sh, long long v_sn, void* k_pages, void* v_pages, void* bounds, const int* block_table,
                    const int* seq_lens, const int* new_lens, const int* positions, const uint64_t* turns, int B, int Hkv,
                    int N, int d, int rot, int interleaved, float magnitude, int page_size, int block, int max_pages,
                    int num_pages, void* stream) {
    if (!k || !v || !k_pages || !v_pages || !block_table || !seq_lens || N < 1) return FA_ERR_INVALID_ARG;
    int st = check_cache(B, Hkv, page_size, bounds ? block : 1, max_pages, num_pages, d);
    if (st != FA_OK) return st;
    if (turns && (st = check_rotation(d, rot, interleaved, magnitude)) != FA_OK) return st;
    if (N > kMaxCacheTokens / 2 || (long long)B * Hkv * N > 0x7FFFFFFFll) return FA_ERR_UNSUPPORTED;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(bounds) ||
        !aligned16(turns) || !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(new_lens) || !aligned4(positions))
        return FA_ERR_ALIGNMENT;
    if ((st = check_strides(&k_sb, &k_sh, &k_sn, B, Hkv, N)) != FA_OK) return st;
    if ((st = check_strides(&v_sb, &v_sh, &v_sn, B, Hkv, N)) != FA_OK) return st;
    PagedAppendLaunch a;
    st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    a.k = k;
    a.v = v;
    a.kb = k_sb;
    a.kh = k_sh;
    a.kn = k_sn;
    a.vb = v_sb;
    a.vh = v_sh;
    a.vn = v_sn;
    a.kp = k_pages;
    a.vp = v_pages;
    a.bounds = bounds;
    a.table = block_table;
    a.lens = seq_lens;
    a.new_lens = new_lens;
    a.positions = positions;
    a.turns = turns;
    a.B = B;
    a.Hkv = Hkv;
    a.N = N;
    a.d = d;
    a.rot = turns ? rot : 0;
    a.interleaved = turns ? interleaved : 0;
    a.page = page_size;
    a.block = bounds ? block : 1;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.magnitude = magnitude;
    return launched(launch_paged_append(a, (cudaStream_t)stream));
}

size_t fa_select_blocks_workspace_bytes(int B, int Hkv, int max_blocks) {
    if (B < 1 || Hkv < 1 || max_blocks < 1 || max_blocks > kMaxCacheTokens || (long long)B * Hkv > (1ll << 24)) return 0;
    return select_workspace(B, Hkv, max_blocks).bytes;
}

int fa_select_blocks(const void* q, const void* bounds, const int* block_table, const int* seq_lens, int* blocks, int B,
                     int Hq, int Hkv, int Nq, int block, int page_blocks, int max_pages, int num_pages, int d, int keep,
                     int first, int recent, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !bounds || !block_table || !seq_lens || !blocks || Hq < 1 || Nq < 1 || page_blocks < 1 || block < 1)
        return FA_ERR_INVALID_ARG;
    if (block > 128 || page_blocks > kMaxCacheTokens / block) return FA_ERR_UNSUPPORTED;
    int st = check_cache(B, Hkv, page_blocks * block, block, max_pages, num_pages, d);
    if (st != FA_OK) return st;
    if (Hq % Hkv || first < 0 || recent < 0 || keep < 1 || (long long)first + recent > keep) return FA_ERR_INVALID_ARG;
    if (Nq > 16 || (long long)B * Hq > (1ll << 24)) return FA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(bounds) || !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(blocks))
        return FA_ERR_ALIGNMENT;
    SelectLaunch a;
    st = device_state(&a.err, &a.num_sms);
    if (st != FA_OK) return st;
    const SelectWorkspace ws = select_workspace(B, Hkv, (long long)max_pages * page_blocks);
    if (!workspace || workspace_bytes < ws.bytes) return FA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    char* base = static_cast<char*>(workspace);
    a.q = q;
    a.bounds = bounds;
    a.table = block_table;
    a.lens = seq_lens;
    a.out = blocks;
    a.exact = base;
    a.scores = reinterpret_cast<uint32_t*>(base + ws.scores);
    a.stride = (long long)max_pages * page_blocks;
    a.B = B;
    a.Hkv = Hkv;
    a.rows = Hq / Hkv * Nq;
    a.block = block;
    a.page_blocks = page_blocks;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.d = d;
    a.keep = keep;
    a.first = first;
    a.recent = recent;
    return launched(launch_select_blocks(a, (cudaStream_t)stream));
}

size_t fa_decode_blocks_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
    if (!rows_sizes_ok(B, Hq, Hkv, Nq, d)) return 0;
    return rows_workspace(B, Hq, Hkv, Nq, d).bytes;
}

int fa_decode_blocks(const void* q, const void* k_pages, const void* v_pages, const int* block_table, const int* seq_lens,
                     const int* blocks, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int page_size, int block, int keep,
                     int max_pages, int num_pages, int d, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (!blocks || keep < 1) return FA_ERR_INVALID_ARG;
    DecodeRowsLaunch a;
    int st = rows_prepare(a, q, k_pages, v_pages, block_table, seq_lens, o, lse, B, Hq, Hkv, Nq, page_size, block, max_pages,
                          num_pages, d, scale);
    if (st != FA_OK) return st;
    if (!aligned4(blocks)) return FA_ERR_ALIGNMENT;
    if ((st = device_state(&a.err, &a.num_sms)) != FA_OK) return st;
    if (!workspace || workspace_bytes < rows_workspace(B, Hq, Hkv, Nq, d).bytes) return FA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    rows_place(a, static_cast<char*>(workspace));
    a.list = blocks;
    a.keep = keep;
    return launched(launch_decode_rows(a, (cudaStream_t)stream));
}

size_t fa_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d) {
    if (!rows_sizes_ok(B, Hq, Hkv, Nq, d)) return 0;
    // the larger of the two forms', whichever the table's width will choose
    return std::max(rows_workspace(B, Hq, Hkv, Nq, d, joint_rows(B, Hq, Hkv, Nq, d, 0)).bytes,
                    rows_workspace(B, Hq, Hkv, Nq, d, 0, prefix_takes_own(B, Hq, Hkv, Nq)).bytes + prefix_workspace(B, Hq, Hkv, Nq, d).bytes +
                        kPrefixSkip);
}

int fa_decode_shared(const void* q, const void* k_pages, const void* v_pages, const int* block_table, const int* seq_lens,
                     const int* shared_len, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int page_size,
                     int max_pages, int num_pages, int d, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (!shared_len) return FA_ERR_INVALID_ARG;
    DecodeRowsLaunch a;
    int st = rows_prepare(a, q, k_pages, v_pages, block_table, seq_lens, o, lse, B, Hq, Hkv, Nq, page_size, 1, max_pages,
                          num_pages, d, scale, Hkv >= 1 && prefix_takes_own(B, Hq, Hkv, Nq));
    if (st != FA_OK) return st;
    if (page_size % 8) return FA_ERR_UNSUPPORTED;  // boxes of 8 rows at least
    if (!aligned4(shared_len)) return FA_ERR_ALIGNMENT;
    if ((st = device_state(&a.err, &a.num_sms)) != FA_OK) return st;
    a.shared = shared_len;
    a.joint = joint_rows(B, Hq, Hkv, Nq, d, (long long)max_pages * page_size);
    if (a.joint) {
        if (!workspace || workspace_bytes < rows_workspace(B, Hq, Hkv, Nq, d, a.joint).bytes) return FA_ERR_WORKSPACE;
        if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
        rows_place(a, static_cast<char*>(workspace));
        return launched(launch_decode_rows(a, (cudaStream_t)stream));
    }
    const PrefixWorkspace pw = prefix_workspace(B, Hq, Hkv, Nq, d);
    const long long most = ((long long)max_pages * page_size + 127) / 128;  // steps of an item
    if ((long long)Hkv * pw.tiles > 0x7FFFFFFFll / most) return FA_ERR_UNSUPPORTED;
    a.merge_only = prefix_takes_own(B, Hq, Hkv, Nq);
    const RowsWorkspace ws = rows_workspace(B, Hq, Hkv, Nq, d, 0, a.merge_only);
    if (!workspace || workspace_bytes < ws.bytes + pw.bytes + kPrefixSkip) return FA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    char* base = static_cast<char*>(workspace) + (reinterpret_cast<uintptr_t>(workspace) & kPrefixSkip);
    rows_place(a, base);
    base += ws.bytes;
    PrefixLaunch p;
    p.q = q;
    p.table = block_table;
    p.lens = seq_lens;
    p.shared = shared_len;
    p.part_o = reinterpret_cast<float*>(base);
    p.part_lse = reinterpret_cast<float*>(base + pw.part_lse);
    p.ends = reinterpret_cast<int*>(base + pw.ends);
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.Nq = Nq;
    p.page = page_size;
    p.box = page_box_rows(page_size);
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.d = d;
    p.tiles = pw.tiles;
    p.tile_rows = pw.tile_rows;
    p.own = a.merge_only;
    p.workers = std::min(a.num_sms, kPrefixMostWorkers);
    if (!p.own) p.workers = (int)std::min<long long>(p.workers, most * Hkv * pw.tiles);  // a step each
    p.scale = scale;
    p.err = a.err;
    p.timeout_ns = g_timeout_ns.load();
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page_size, (cuuint64_t)Hkv, (cuuint64_t)num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)page_size * d * 2, (cuuint64_t)Hkv * page_size * d * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1};
    if (make_map_nd(&p.map_k, k_pages, 4, dims, strides, box) || make_map_nd(&p.map_v, v_pages, 4, dims, strides, box))
        return FA_ERR_CUDA;
    a.pre_o = p.part_o;
    a.pre_lse = p.part_lse;
    a.pre_ends = p.ends;
    a.pre_workers = p.workers;
    a.pre_tiles = p.tiles;
    a.pre_rows = p.tile_rows;
    st = launched(launch_prefix(p, a, (cudaStream_t)stream));
    return st != FA_OK ? st : launched(launch_decode_rows(a, (cudaStream_t)stream));
}

int fa_selftest_wait_timeout(uint64_t timeout_ns, void* stream) {
    if (timeout_ns < 1000ull || timeout_ns > 1000000000ull) return FA_ERR_INVALID_ARG;
    DevError* err = nullptr;
    int st = device_state(&err, nullptr);
    if (st != FA_OK) return st;
    selftest_wait_kernel<<<1, 32, 0, (cudaStream_t)stream>>>(err, timeout_ns);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_get_last_device_error(void* stream, int* detail) {
    if (detail)
        for (int i = 0; i < 4; ++i) detail[i] = 0;
    DevError* err = nullptr;
    if (device_state(&err, nullptr) != FA_OK) return FA_ERR_CUDA;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return FA_ERR_CUDA;
    DevError h;
    if (cudaMemcpy(&h, err, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return FA_ERR_CUDA;
    if (h.code != 0) {
        DevError z = {0, 0, 0, 0};
        if (cudaMemcpy(err, &z, sizeof(z), cudaMemcpyHostToDevice) != cudaSuccess) return FA_ERR_CUDA;
    }
    if (detail) {
        detail[0] = h.code;
        detail[1] = h.site;
        detail[2] = h.block;
        detail[3] = h.aux;
    }
    return h.code;  // FA_OK, or the first code a kernel recorded
}

}  // extern "C"

// ---------------------------------------------------------------- decode without a workspace
// fa_decode_noalloc: the split partials live in one fixed array compiled into
// the library, for callers that may not allocate device memory (see fa.h).
// In host code the name of the array is only a stand-in; its device address
// comes from cudaGetSymbolAddress, looked up once per device with that device
// current, and is what the kernels receive.
static __device__ __align__(256) unsigned char g_fa_decode_scratch[FA_DECODE_NOALLOC_SCRATCH_BYTES];

namespace {
std::mutex g_scratch_mu;
void* g_scratch_addr[fa::kMaxDevices] = {};
}  // namespace

extern "C" int fa_decode_noalloc(const void* q, const void* kcache, const void* vcache, void* o, float* lse,
                                 int B, int H, int Nk, int d, float scale, int num_splits, void* stream) {
    if (!q || !kcache || !vcache || !o) return FA_ERR_INVALID_ARG;
    if (!scale_ok(scale) || num_splits > 256) return FA_ERR_INVALID_ARG;
    int st = check_shape(B, H, 1, Nk, d);
    if (st != FA_OK) return st;
    if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(o) ||
        (lse && !aligned16(lse)))
        return FA_ERR_ALIGNMENT;
    int splits = num_splits <= 0 ? decode_auto_splits(Nk) : num_splits;  // the rule of fa_decode
    if (num_splits <= 0 && !contiguous_on_mma(Nk, d)) {
        st = decode_wave_splits(B, H, Nk, d, &splits);
        if (st != FA_OK) return st;
    }
    if (decode_ws_bytes(B, H, d, splits) > FA_DECODE_NOALLOC_SCRATCH_BYTES) return FA_ERR_WORKSPACE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
    void* scratch = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        if (!g_scratch_addr[dev]) {
            void* addr = nullptr;
            if (cudaGetSymbolAddress(&addr, g_fa_decode_scratch) != cudaSuccess || !addr) return FA_ERR_CUDA;
            g_scratch_addr[dev] = addr;
        }
        scratch = g_scratch_addr[dev];
    }
    if (contiguous_on_mma(Nk, d))
        return launch_contiguous_on_mma(q, kcache, vcache, o, lse, B, H, Nk, d, scale, splits,
                                        static_cast<float*>(scratch), stream);
    DecodeLaunch a;
    a.q = q;
    a.kc = kcache;
    a.vc = vcache;
    a.o = o;
    a.lse = lse;
    a.part_o = static_cast<float*>(scratch);
    a.part_lse = a.part_o + (size_t)B * H * splits * d;  // same layout as the fa_decode workspace
    a.B = B;
    a.H = H;
    a.Nk = Nk;
    a.d = d;
    a.splits = splits;
    a.chunk = (Nk + splits - 1) / splits;
    a.scale = scale;
    return launch_decode(a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
